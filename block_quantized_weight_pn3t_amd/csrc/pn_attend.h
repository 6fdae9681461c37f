// pn_attend.h -- attention of a step's tokens over a shared prefix and each sequence's own tokens,
// read from the microscaled cache, on gfx950.
//
// out = sum_j w_j v_j / sum_j w_j, w_j = exp(scale * q.k_j). One pass over the tokens: a running
// maximum m, l = sum exp(s - m) and O = sum exp(s - m) v, rescaled when m grows; partial results of
// disjoint token ranges join as m = max m_i, l = sum l_i e^(m_i - m), O likewise.
//
// A wave holds RT tiles of 16 query rows (a row is one query token and head of a KV head's group;
// in the prefix the rows of all sequences stand in one list) and walks records of 32 tokens:
//   S^T = K Q^T  16x16x32 bf16 matrix instructions, tokens as rows: lane (i, g) = (lane % 16,
//                lane / 16) takes 16-channel pieces of token i straight from the record (16 bytes a
//                lane, a wave's load is one contiguous run), converted exactly to bf16 with the
//                block's exponent by one instruction a pair. A lane's results are four tokens
//                (4g .. 4g + 3 of each half) of query row i.
//   O^T += V^T P^T  the same lane supplies P for exactly those tokens, so the weights never leave
//                their registers; V's dwords hold four channels of one token, and a byte permute of
//                two converted tokens makes the pairs along the tokens that the instruction takes.
//                A lane's results belong to row i again, so the rescaling by exp(m - m') is its own
//                row's and needs no exchange; only m takes two lane swaps a record.
// No LDS and no barrier until the end: the four waves of a workgroup take every fourth record of the
// workgroup's token range and join their results through LDS. The range is one of `splits` of a
// sequence (or of the prefix), and a second kernel joins those.
#pragma once

#include <math.h>

#include <algorithm>

#include "pn_cache.h"

namespace pn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct AttendArgs {
    CacheView c;
    int type, B, Q, Hq, G;  // G query heads a KV head
    const void *q;
    int64_t q_seq, q_tok, q_head;
    int q_vec;     // q can be loaded 16 bytes at a time
    float scale;   // |scale| * log2(e), at least the least normal number
    int neg;       // scale < 0: q is negated as it is loaded
    const int32_t *table, *lens, *q_lens, *prefix_table;
    int64_t table_stride;
    int table_width, prefix_len;
    int prefix_splits, prefix_blocks;  // token ranges and row blocks of the prefix (0 without one)
    int own_splits, own_blocks;        // token ranges of a sequence and row blocks of a KV head
    int direct;                        // one range in all: write out, nothing to join
    float *part;                       // [range][row][D]
    float2 *part_ml;                   // [range][row]: maximum (log2 units) and sum
    void *out;
    float *lse;
};

// Tokens first..last of range `split`: whole records, spread evenly.
struct Range {
    int begin, end;  // records
};
__device__ __forceinline__ Range split_range(int tokens, int splits, int split)
{
    const int records = (tokens + kTile - 1) / kTile;
    const int each = (records + splits - 1) / splits;
    return Range{min(records, each * split), min(records, each * (split + 1))};
}
// How many of the ranges hold a record.
__device__ __forceinline__ int live_ranges(int tokens, int splits)
{
    const int records = (tokens + kTile - 1) / kTile;
    const int each = (records + splits - 1) / splits;
    return each ? (records + each - 1) / each : 0;
}

// Own tokens and query tokens of sequence b, as the tables allow.
__device__ __forceinline__ int own_tokens(const AttendArgs &A, int b)
{
    return min(max(A.lens[b], 0), A.table_width << A.c.page_shift);
}
__device__ __forceinline__ int query_tokens(const AttendArgs &A, int b)
{
    return A.q_lens ? min(max(A.q_lens[b], 0), A.Q) : A.Q;
}

__device__ __forceinline__ float load_elem(int type, const void *p, int64_t at)
{
    return type == PN_F32    ? reinterpret_cast<const float *>(p)[at]
           : type == PN_BF16 ? (float)reinterpret_cast<const __bf16 *>(p)[at]
                             : (float)reinterpret_cast<const _Float16 *>(p)[at];
}

__device__ __forceinline__ void store_elem(int type, void *p, int64_t at, float x)
{
    if (type == PN_F32)
        reinterpret_cast<float *>(p)[at] = x;
    else if (type == PN_BF16)
        reinterpret_cast<__bf16 *>(p)[at] = (__bf16)x;
    else
        reinterpret_cast<_Float16 *>(p)[at] = (_Float16)x;
}

// Eight channels of q as NT bf16 parts: the value rounded, then what that left. bf16 q has one part
// (exact), fp16 two (exact: 11 bits), fp32 two (2^-16 relative at most).
template <int NT>
__device__ __forceinline__ void load_q8(const AttendArgs &A, int64_t at, bool live,
                                        bf16x8_t (&part)[NT])
{
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; j++)
        x[j] = 0.0f;
    if (live) {
        if (A.q_vec && A.type == PN_F32) {
            const f32x4_t *p = reinterpret_cast<const f32x4_t *>(reinterpret_cast<const float *>(A.q) + at);
            const f32x4_t a = p[0], b = p[1];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                x[j] = a[j];
                x[4 + j] = b[j];
            }
        } else if (A.q_vec && A.type == PN_BF16) {
            const bf16x8_t a = *reinterpret_cast<const bf16x8_t *>(reinterpret_cast<const __bf16 *>(A.q) + at);
#pragma unroll
            for (int j = 0; j < 8; j++)
                x[j] = (float)a[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++)
                x[j] = load_elem(A.type, A.q, at + j);
        }
    }
#pragma unroll
    for (int j = 0; j < 8; j++) {
        float v = A.neg ? -x[j] : x[j];
#pragma unroll
        for (int t = 0; t < NT; t++) {
            part[t][j] = (__bf16)v;
            v -= (float)part[t][j];
        }
    }
}

__device__ __forceinline__ uint32_t dword(const uint4 &v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

__device__ __forceinline__ float exp_bits(uint32_t w) { return __builtin_bit_cast(float, w); }

// A pair of codes as bf16: the pair at 16-bit (8-bit codes) or 8-bit (4-bit codes) position SEL of w.
// The instruction takes the power of two from bits 23..30 of `s` and ignores its other bits, so one
// shift brings any byte of an exponent word into place.
template <int FMT, int SEL>
__device__ __forceinline__ uint32_t pair(uint32_t w, float s)
{
    if constexpr (FMT == PN_CACHE_MXFP8)
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, SEL != 0));
    else
        return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, SEL));
}

__device__ __forceinline__ f32x4_t mfma(bf16x8_t a, bf16x8_t b, f32x4_t c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ float over_groups_max(float v)
{
    float a = v, b = v;
    swap32(a, b);
    v = fmaxf(a, b);
    a = b = v;
    swap16(a, b);
    return fmaxf(a, b);
}
__device__ __forceinline__ float over_groups_sum(float v)
{
    float a = v, b = v;
    swap32(a, b);
    v = a + b;
    a = b = v;
    swap16(a, b);
    return a + b;
}

// A record's K (or V) half in a lane's registers.
template <int FMT, int D>
struct KReg {
    static constexpr int N = (FMT == PN_CACHE_MXFP8 ? 2 : 1) * Rec<FMT, D>::NP;
    uint4 w[N];
    uint32_t e[2];  // byte 2p + a: the exponent of chunk p, half a (this lane's token and block)
};
template <int FMT, int D>
struct VReg {
    static constexpr int N = KReg<FMT, D>::N;
    uint4 w[N];
    uint32_t e[2 * Rec<FMT, D>::NP];  // word 2p + a: the exponents of this lane's four tokens
};

template <int FMT, int D>
__device__ __forceinline__ void load_k(const uint8_t *rec, int lane, KReg<FMT, D> &k)
{
    constexpr int NP = Rec<FMT, D>::NP;
#pragma unroll
    for (int n = 0; n < KReg<FMT, D>::N; n++)
        k.w[n] = *reinterpret_cast<const uint4 *>(rec + (n * 64 + lane) * 16);
    const uint8_t *e = rec + Rec<FMT, D>::KE + ((lane >> 5) * 16 + (lane & 15)) * NP * 2;
    if constexpr (NP == 1) {
        k.e[0] = *reinterpret_cast<const uint16_t *>(e);
    } else if constexpr (NP == 2) {
        k.e[0] = *reinterpret_cast<const uint32_t *>(e);
    } else {
        const uint2 t = *reinterpret_cast<const uint2 *>(e);
        k.e[0] = t.x;
        k.e[1] = t.y;
    }
}

template <int FMT, int D>
__device__ __forceinline__ void load_v(const uint8_t *rec, int lane, VReg<FMT, D> &v)
{
    constexpr int NP = Rec<FMT, D>::NP;
#pragma unroll
    for (int n = 0; n < VReg<FMT, D>::N; n++)
        v.w[n] = *reinterpret_cast<const uint4 *>(rec + Rec<FMT, D>::V + (n * 64 + lane) * 16);
    const uint2 *e = reinterpret_cast<const uint2 *>(
        rec + Rec<FMT, D>::VE + (((lane >> 3) & 1) * 4 + (lane >> 4)) * NP * 8);
#pragma unroll
    for (int p = 0; p < NP; p++) {
        const uint2 t = e[p];
        v.e[2 * p] = t.x;
        v.e[2 * p + 1] = t.y;
    }
}

// Eight channels (piece half J) of chunk p of this lane's token of half a.
template <int FMT, int D>
__device__ __forceinline__ bf16x8_t k_frag(const KReg<FMT, D> &k, int p, int a, int j)
{
    const int byte = 2 * p + a;
    const uint32_t w = k.e[byte >> 2];
    const int b = byte & 3;
    const float s = exp_bits(b == 0 ? w << 23 : b == 1 ? w << 15 : b == 2 ? w << 7 : w >> 1);
    uint32_t r[4];
    if constexpr (FMT == PN_CACHE_MXFP8) {
        const uint32_t lo = dword(k.w[2 * p + a], 2 * j), hi = dword(k.w[2 * p + a], 2 * j + 1);
        r[0] = pair<FMT, 0>(lo, s);
        r[1] = pair<FMT, 1>(lo, s);
        r[2] = pair<FMT, 0>(hi, s);
        r[3] = pair<FMT, 1>(hi, s);
    } else {
        const uint32_t lo = dword(k.w[p], 2 * a + j);
        r[0] = pair<FMT, 0>(lo, s);
        r[1] = pair<FMT, 1>(lo, s);
        r[2] = pair<FMT, 2>(lo, s);
        r[3] = pair<FMT, 3>(lo, s);
    }
    return __builtin_bit_cast(bf16x8_t, make_uint4(r[0], r[1], r[2], r[3]));
}

// Chunk p of V as four operands: operand n holds channel 64p + 4i + n of this lane's eight tokens.
template <int FMT, int D>
__device__ __forceinline__ void v_frags(const VReg<FMT, D> &v, int p, bf16x8_t (&f)[4])
{
    uint32_t r[4][4];
#pragma unroll
    for (int a = 0; a < 2; a++) {
        const uint32_t w = v.e[2 * p + a];
        const float s[4] = {exp_bits(w << 23), exp_bits(w << 15), exp_bits(w << 7), exp_bits(w >> 1)};
        uint32_t c01[4], c23[4];
        if constexpr (FMT == PN_CACHE_MXFP8) {
#pragma unroll
            for (int t = 0; t < 4; t++) {
                c01[t] = pair<FMT, 0>(dword(v.w[2 * p + a], t), s[t]);
                c23[t] = pair<FMT, 1>(dword(v.w[2 * p + a], t), s[t]);
            }
        } else {
#pragma unroll
            for (int t = 0; t < 4; t += 2) {
                const uint32_t d = dword(v.w[p], 2 * a + t / 2);
                c01[t] = pair<FMT, 0>(d, s[t]);
                c23[t] = pair<FMT, 1>(d, s[t]);
                c01[t + 1] = pair<FMT, 2>(d, s[t + 1]);
                c23[t + 1] = pair<FMT, 3>(d, s[t + 1]);
            }
        }
#pragma unroll
        for (int t = 0; t < 2; t++) {
            r[0][2 * a + t] = __builtin_amdgcn_perm(c01[2 * t + 1], c01[2 * t], 0x05040100);
            r[1][2 * a + t] = __builtin_amdgcn_perm(c01[2 * t + 1], c01[2 * t], 0x07060302);
            r[2][2 * a + t] = __builtin_amdgcn_perm(c23[2 * t + 1], c23[2 * t], 0x05040100);
            r[3][2 * a + t] = __builtin_amdgcn_perm(c23[2 * t + 1], c23[2 * t], 0x07060302);
        }
    }
#pragma unroll
    for (int n = 0; n < 4; n++)
        f[n] = __builtin_bit_cast(bf16x8_t, make_uint4(r[n][0], r[n][1], r[n][2], r[n][3]));
}

// Token (a, t) of this lane's eight, chunk p: zeros.
template <int FMT, int D>
__device__ __forceinline__ void v_clear(VReg<FMT, D> &v, int p, int a, int t)
{
    uint4 &w = v.w[FMT == PN_CACHE_MXFP8 ? 2 * p + a : p];
    const int d = FMT == PN_CACHE_MXFP8 ? t : 2 * a + t / 2;
    const uint32_t keep = FMT == PN_CACHE_MXFP8 ? 0u : t & 1 ? 0x0000FFFFu : 0xFFFF0000u;
    if (d == 0)
        w.x &= keep;
    else if (d == 1)
        w.y &= keep;
    else if (d == 2)
        w.z &= keep;
    else
        w.w &= keep;
    v.e[2 * p + a] &= ~(255u << (8 * t));
}

// NaN blocks in a record that some rows see only in part: a weight of zero must not meet them. They
// are taken out of V, and what they do to the rows that see them is done here: a product of "is NaN"
// with "is seen" counts, for each row and channel, the NaNs that belong to its sum.
template <int FMT, int D, int RT>
__device__ __forceinline__ void v_nan_apart(VReg<FMT, D> &v, const f32x4_t (&s)[RT][2],
                                            f32x4_t (&O)[RT][Rec<FMT, D>::NP][4])
{
    constexpr int NP = Rec<FMT, D>::NP;
#pragma unroll
    for (int p = 0; p < NP; p++) {
        bf16x8_t bad;
#pragma unroll
        for (int a = 0; a < 2; a++)
#pragma unroll
            for (int t = 0; t < 4; t++) {
                const bool nan = ((v.e[2 * p + a] >> (8 * t)) & 255u) == 255u;
                bad[4 * a + t] = (__bf16)(nan ? 1.0f : 0.0f);
                if (nan)
                    v_clear<FMT, D>(v, p, a, t);
            }
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
            bf16x8_t seen;
#pragma unroll
            for (int a = 0; a < 2; a++)
#pragma unroll
                for (int r = 0; r < 4; r++)
                    seen[4 * a + r] = (__bf16)(s[rt][a][r] == -INFINITY ? 0.0f : 1.0f);
            const f32x4_t count = mfma(bad, seen, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
            for (int n = 0; n < 4; n++)
#pragma unroll
                for (int r = 0; r < 4; r++)
                    O[rt][p][n][r] = count[r] > 0.0f ? __builtin_nanf("") : O[rt][p][n][r];
        }
    }
}

// One workgroup's share: rows [row0, row0 + 16 RT) of KV head h over range `split` of a sequence's
// own tokens (OWN) or of the prefix.
template <int FMT, int D, int NT, int RT, bool OWN>
__device__ __forceinline__ void attend_part(const AttendArgs &A, int split, int b0, int h, int row0,
                                            float *lds)
{
    constexpr int NP = Rec<FMT, D>::NP;
    typedef Rec<FMT, D> R;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;

    const int nrows = (OWN ? 1 : A.B) * A.Q * A.G;
    const int tokens = OWN ? own_tokens(A, b0) : A.prefix_len;
    const int nq = OWN ? query_tokens(A, b0) : A.Q;
    const int least = OWN ? tokens - nq + 1 : tokens;  // the tokens below are seen by every row
    const Range range = split_range(tokens, OWN ? A.own_splits : A.prefix_splits, split);
    if (range.begin >= range.end && !A.direct)
        return;

    // this lane's rows: where they are in q and out, and up to which token they see
    int limit[RT];
    bf16x8_t q[RT][NP][2][NT];
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        const int row = row0 + 16 * rt + i16;
        const bool live = row < nrows;
        const int r = live ? row : 0;
        const int qt = r / A.G;  // query token, counted over all sequences in the prefix
        const int b = OWN ? b0 : qt / A.Q, i = OWN ? qt : qt - b * A.Q;
        limit[rt] = !OWN ? tokens : i < nq ? min(tokens, tokens - nq + i + 1) : 0;
        const int64_t at = b * A.q_seq + i * A.q_tok + (h * A.G + r - qt * A.G) * A.q_head;
#pragma unroll
        for (int p = 0; p < NP; p++)
#pragma unroll
            for (int j = 0; j < 2; j++)
                load_q8<NT>(A, at + 64 * p + 16 * g + 8 * j, live, q[rt][p][j]);
    }

    f32x4_t O[RT][NP][4];
    float m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        m[rt] = -INFINITY;
        l[rt] = 0.0f;
#pragma unroll
        for (int p = 0; p < NP; p++)
#pragma unroll
            for (int n = 0; n < 4; n++)
                O[rt][p][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }

    const int32_t *table = OWN ? A.table + b0 * A.table_stride : A.prefix_table;
    const int tshift = A.c.page_shift - 5;  // log2 of the records a page has
    auto page_of = [&](int t) {
        const int64_t page = table[t >> tshift];
        return page < 0 ? (int64_t)0 : min(page, A.c.pages - 1);
    };
    auto record = [&](int64_t page, int t) -> const uint8_t * {
        return A.c.data + (((page * A.c.heads + h) << tshift) + (t & ((1 << tshift) - 1))) * R::BYTES;
    };

    KReg<FMT, D> kr;
    VReg<FMT, D> vr;
    int t = range.begin + wave;
    int64_t next_page = 0;
    if (t < range.end) {
        const uint8_t *rec = record(page_of(t), t);
        load_k<FMT, D>(rec, lane, kr);
        load_v<FMT, D>(rec, lane, vr);
        if (t + 4 < range.end)
            next_page = page_of(t + 4);
    }
    for (; t < range.end; t += 4) {
        const bool more = t + 4 < range.end;
        const uint8_t *next = record(next_page, t + 4);

        // scores of 2 x 16 tokens
        f32x4_t s[RT][2];
#pragma unroll
        for (int rt = 0; rt < RT; rt++)
            s[rt][0] = s[rt][1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int p = 0; p < NP; p++)
#pragma unroll
            for (int a = 0; a < 2; a++)
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    const bf16x8_t kf = k_frag<FMT, D>(kr, p, a, j);
#pragma unroll
                    for (int rt = 0; rt < RT; rt++)
#pragma unroll
                        for (int n = 0; n < NT; n++)
                            s[rt][a] = mfma(kf, q[rt][p][j][n], s[rt][a]);
                }
        if (more) {
            load_k<FMT, D>(next, lane, kr);
            if (t + 8 < range.end)
                next_page = page_of(t + 8);
        }

        // the record holds tokens that some row does not see: those count nothing, and what lies
        // past the sequence's end (anything at all) must not meet a weight of zero as NaN
        bool nan_hidden = false;
        if ((t + 1) * kTile > least) {
            const int first = t * kTile + 4 * g;
#pragma unroll
            for (int a = 0; a < 2; a++)
#pragma unroll
                for (int r = 0; r < 4; r++) {
#pragma unroll
                    for (int rt = 0; rt < RT; rt++)
                        if (first + 16 * a + r >= limit[rt])
                            s[rt][a][r] = -INFINITY;
                    if (first + 16 * a + r >= tokens) {
#pragma unroll
                        for (int p = 0; p < NP; p++) {
                            v_clear<FMT, D>(vr, p, a, r);
                        }
                    }
                }
            if (OWN) {  // a NaN block of a token that only some rows see
                bool any = false;
#pragma unroll
                for (int p = 0; p < 2 * NP; p++)
#pragma unroll
                    for (int r = 0; r < 4; r++)
                        any |= ((vr.e[p] >> (8 * r)) & 255u) == 255u;
                nan_hidden = __any(any);
            }
        }

        uint32_t pw[RT][NT][4];
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
            float top = fmaxf(fmaxf(fmaxf(s[rt][0][0], s[rt][0][1]), fmaxf(s[rt][0][2], s[rt][0][3])),
                              fmaxf(fmaxf(s[rt][1][0], s[rt][1][1]), fmaxf(s[rt][1][2], s[rt][1][3])));
            top = over_groups_max(top) * A.scale;
            // the maximum may lag by 2^8 of growth: weights up to 256 lose nothing, and most
            // records need no rescaling
            if (__any(top > m[rt] + 8.0f)) {
                const float now = fmaxf(m[rt], top);
                const float f = now == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[rt] - now);
                m[rt] = now;
                l[rt] *= f;
#pragma unroll
                for (int p = 0; p < NP; p++)
#pragma unroll
                    for (int n = 0; n < 4; n++)
                        O[rt][p][n] *= f;
            }
            const float base = m[rt] == -INFINITY ? 0.0f : -m[rt];
            float w[8];
#pragma unroll
            for (int a = 0; a < 2; a++)
#pragma unroll
                for (int r = 0; r < 4; r++)
                    w[4 * a + r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][a][r], A.scale, base));
            l[rt] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int r = 0; r < 4; r++) {
                    const bf16x2_t v = {(__bf16)w[2 * r], (__bf16)w[2 * r + 1]};
                    pw[rt][n][r] = __builtin_bit_cast(uint32_t, v);
                    if (n + 1 < NT) {
                        w[2 * r] -= (float)v.x;
                        w[2 * r + 1] -= (float)v.y;
                    }
                }
        }

        if (nan_hidden)
            v_nan_apart<FMT, D, RT>(vr, s, O);
#pragma unroll
        for (int p = 0; p < NP; p++) {
            bf16x8_t vf[4];
            v_frags<FMT, D>(vr, p, vf);
#pragma unroll
            for (int n = 0; n < 4; n++)
#pragma unroll
                for (int rt = 0; rt < RT; rt++)
#pragma unroll
                    for (int e = 0; e < NT; e++)
                        O[rt][p][n] = mfma(vf[n],
                                           __builtin_bit_cast(bf16x8_t, make_uint4(pw[rt][e][0], pw[rt][e][1],
                                                                                   pw[rt][e][2], pw[rt][e][3])),
                                           O[rt][p][n]);
        }
        if (more)
            load_v<FMT, D>(next, lane, vr);
    }

    // join the four waves, a tile of 16 rows at a time: lds holds their O, then m and l
    constexpr int PAD = D + 4;
    float *const mls = lds + 4 * 16 * PAD;  // [wave][row][2]
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        const float lsum = over_groups_sum(l[rt]);
        if (rt > 0)
            __syncthreads();
#pragma unroll
        for (int p = 0; p < NP; p++)
#pragma unroll
            for (int r = 0; r < 4; r++)
                *reinterpret_cast<f32x4_t *>(lds + (wave * 16 + i16) * PAD + 64 * p + 16 * g + 4 * r) =
                    f32x4_t{O[rt][p][0][r], O[rt][p][1][r], O[rt][p][2][r], O[rt][p][3][r]};
        if (g == 0) {
            mls[(wave * 16 + i16) * 2] = m[rt];
            mls[(wave * 16 + i16) * 2 + 1] = lsum;
        }
        __syncthreads();
        // thread = row * 16 + channel group
        const int jr = threadIdx.x >> 4, cg = threadIdx.x & 15;
        const int row = row0 + 16 * rt + jr;
        if (row < nrows) {
            float top = -INFINITY, sum = 0.0f, f[4];
            bool saw[4];
#pragma unroll
            for (int w = 0; w < 4; w++)
                top = fmaxf(top, mls[(w * 16 + jr) * 2]);
#pragma unroll
            for (int w = 0; w < 4; w++) {
                // l = 0 only where a wave saw no token (l is NaN where its scores are)
                const float lw = mls[(w * 16 + jr) * 2 + 1];
                saw[w] = lw != 0.0f;
                f[w] = saw[w] ? __builtin_amdgcn_exp2f(mls[(w * 16 + jr) * 2] - top) : 0.0f;
                sum += f[w] * lw;
            }
            const int qt = row / A.G;
            const int b = OWN ? b0 : qt / A.Q, i = OWN ? qt : qt - b * A.Q;
            const int64_t orow = ((int64_t)b * A.Q + i) * A.Hq + h * A.G + (row - qt * A.G);
            const int64_t rows = (int64_t)A.B * A.Q * A.Hq;
            const int64_t slot = (OWN ? A.prefix_splits : 0) + split;
            if (A.direct && i >= nq)
                sum = 0.0f;  // not a query token of this sequence
            const bool none = sum == 0.0f;
            const float inv = 1.0f / sum;
#pragma unroll
            for (int p = 0; p < NP; p++) {
                f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int w = 0; w < 4; w++)
                    if (saw[w])
                        v += f[w] * *reinterpret_cast<const f32x4_t *>(lds + (w * 16 + jr) * PAD + 64 * p + 4 * cg);
                const int64_t at = orow * D + 64 * p + 4 * cg;
                if (A.direct) {
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        store_elem(A.type, A.out, at + e, none ? 0.0f : v[e] * inv);
                } else {
                    *reinterpret_cast<f32x4_t *>(A.part + slot * rows * D + at) = v;
                }
            }
            if (cg == 0) {
                if (!A.direct)
                    A.part_ml[slot * rows + orow] = make_float2(top, sum);
                else if (A.lse)
                    A.lse[orow] = none ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
            }
        }
    }
}

// Workgroups: first the prefix's [row block][KV head and range], then [range][sequence][row block][KV
// head] of the own tokens. RP, RO: tiles of 16 rows a wave holds in the prefix (0: no prefix) and in
// the own tokens.
template <int FMT, int D, int NT, int RP, int RO>
__global__ void __launch_bounds__(256) attend_kernel(AttendArgs A)
{
    extern __shared__ float lds[];
    int id = blockIdx.x;
    if constexpr (RP > 0) {
        const int each = A.c.heads * A.prefix_splits;
        if (id < each * A.prefix_blocks) {
            const int block = id / each, rest = id - block * each;
            const int split = rest / A.c.heads, h = rest - split * A.c.heads;
            attend_part<FMT, D, NT, RP, false>(A, split, 0, h, block * 16 * RP, lds);
            return;
        }
        id -= each * A.prefix_blocks;
    }
    const int h = id % A.c.heads;
    id /= A.c.heads;
    const int block = id % A.own_blocks;
    id /= A.own_blocks;
    const int b = id % A.B;
    attend_part<FMT, D, NT, RO, true>(A, id / A.B, b, h, block * 16 * RO, lds);
}

// Joins the ranges of one row: a wave a row, lane = channels D / 64 * lane ...
template <int D>
__global__ void __launch_bounds__(256) attend_join_kernel(AttendArgs A)
{
    constexpr int C = D / 64;
    typedef float vec __attribute__((ext_vector_type(C)));
    const int lane = threadIdx.x & 63;
    const int64_t rows = (int64_t)A.B * A.Q * A.Hq;
    const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (row >= rows)
        return;
    const int qt = (int)(row / A.Hq), b = qt / A.Q, i = qt - b * A.Q;
    int np = live_ranges(A.prefix_len, A.prefix_splits ? A.prefix_splits : 1);
    int n = np + live_ranges(own_tokens(A, b), A.own_splits);
    if (i >= query_tokens(A, b))
        n = np = 0;
    const auto slot = [&](int k) -> int64_t { return k < np ? k : A.prefix_splits + k - np; };
    float top = -INFINITY;
    for (int k = lane; k < n; k += 64)
        top = fmaxf(top, A.part_ml[slot(k) * rows + row].x);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor(top, o, 64));
    float sum = 0.0f;
    vec acc = {};
    for (int k0 = 0; k0 < n; k0 += 64) {
        float f = 0.0f;
        if (k0 + lane < n) {
            const float2 ml = A.part_ml[slot(k0 + lane) * rows + row];
            f = ml.y != 0.0f ? __builtin_amdgcn_exp2f(ml.x - top) : 0.0f;
            sum += f * ml.y;
        }
        const int most = min(64, n - k0);
#pragma unroll 8
        for (int k = 0; k < most; k++) {
            const float fk = __builtin_bit_cast(
                float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), k));
            const vec o = *reinterpret_cast<const vec *>(A.part + (slot(k0 + k) * rows + row) * D + C * lane);
            acc += fk * o;
        }
    }
    sum = wave_sum(sum);
    const bool none = sum == 0.0f;
    const float inv = 1.0f / sum;
#pragma unroll
    for (int e = 0; e < C; e++)
        store_elem(A.type, A.out, row * D + C * lane + e, none ? 0.0f : acc[e] * inv);
    if (lane == 0 && A.lse)
        A.lse[row] = none ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <int FMT, int D, int NT, int RP, int RO>
static int launch_attend(const AttendArgs &A, hipStream_t s)
{
    constexpr auto kern = attend_kernel<FMT, D, NT, RP, RO>;
    constexpr int bytes = (4 * 16 * (D + 4) + 4 * 16 * 2) * 4;
    if (!lds_limit_once<kern>(bytes))
        return PN_ERR_HIP;
    const int64_t grid = (int64_t)A.c.heads * A.prefix_splits * A.prefix_blocks +
                         (int64_t)A.own_splits * A.B * A.own_blocks * A.c.heads;
    if (grid > INT32_MAX)
        return PN_ERR_SHAPE;
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(256), bytes, s, A);
    const int st = launch_status();
    if (st != PN_OK || A.direct)
        return st;
    const int64_t rows = (int64_t)A.B * A.Q * A.Hq;
    hipLaunchKernelGGL((attend_join_kernel<D>), dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, s, A);
    return launch_status();
}

// rp, ro: the rows a wave holds, as attend_cut chose them
template <int FMT, int D, int NT>
static int launch_rows(const AttendArgs &A, int rp, int ro, hipStream_t s)
{
    constexpr int MOST = D == 256 || NT == 2 ? 2 : 4;
    if (ro == 1)
        return rp == 0   ? launch_attend<FMT, D, NT, 0, 1>(A, s)
               : rp == 1 ? launch_attend<FMT, D, NT, 1, 1>(A, s)
                         : launch_attend<FMT, D, NT, MOST, 1>(A, s);
    return rp == 0 ? launch_attend<FMT, D, NT, 0, 2>(A, s) : launch_attend<FMT, D, NT, MOST, 2>(A, s);
}

// Launches format FMT, one source file each.
template <int FMT>
int launch_format(const AttendArgs &A, int dim, bool two, int rp, int ro, hipStream_t s);

#define PN_ATTEND_FORMAT(FMT)                                                                      \
    template <>                                                                                    \
    int launch_format<FMT>(const AttendArgs &A, int dim, bool two, int rp, int ro, hipStream_t s)  \
    {                                                                                              \
        switch (dim) {                                                                             \
        case 64: return two ? launch_rows<FMT, 64, 2>(A, rp, ro, s) : launch_rows<FMT, 64, 1>(A, rp, ro, s); \
        case 128: return two ? launch_rows<FMT, 128, 2>(A, rp, ro, s) : launch_rows<FMT, 128, 1>(A, rp, ro, s); \
        default: return two ? launch_rows<FMT, 256, 2>(A, rp, ro, s) : launch_rows<FMT, 256, 1>(A, rp, ro, s); \
        }                                                                                          \
    }

}  // namespace pn
