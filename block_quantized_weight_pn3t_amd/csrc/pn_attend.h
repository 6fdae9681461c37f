// pn_attend.h -- attention of a step's tokens over a shared prefix and each sequence's own tokens,
// read from the microscaled cache, on gfx950.
//
// out = sum_j w_j v_j / sum_j w_j, w_j = exp(scale * q.k_j). One pass over the tokens: a reference m
// near the running maximum, l = sum exp(s - m) and O = sum exp(s - m) v, rescaled when m moves; partial results of
// disjoint token ranges join as m = max m_i, l = sum l_i e^(m_i - m), O likewise.
//
// Tiles are 16 query rows (a row is one query token and head of a KV head's group; in the prefix the
// rows of all sequences stand in one list) by records of 32 tokens:
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
// (The block-scaled 8-bit matrix instructions would take K's codes as they are, but align the 128
// products of a sum to 13 bits below the largest: measured, 2^8 + 127 * 2^-6 gives 2^8.)
//
// Two kinds of workgroup, both of eight waves, two a SIMD: a single wave issues a vector instruction
// every 7 clocks here, two together every 4.6.
//   stream  few rows: memory bound. A wave has one tile of rows, q in LDS, and every (8 / tiles)-th
//           record of the workgroup's token range, from memory straight to registers; at the end the
//           waves of a row tile join through LDS.
//   shared  the prefix under more than 64 rows: bound by the matrix and vector instructions and LDS
//           reads together. All waves walk the same records, each with its own 16 to 48 rows.
//           Converting a record once a wave would cost as much as its products, so it is converted once
//           a workgroup: each wave takes half a chunk of 64 channels of K and of V and puts the operands
//           into LDS, K two stages ahead and V one (rings of three and two, one barrier a stage).
// A workgroup's token range is one of `splits` of its sequence's (or the prefix's), and a second
// kernel joins those.
//
// Measured: four query tokens of 24 heads over 130,077 of 4 x 256 channels, fp32, 8-bit codes (stream):
// 62 us and 4.8 of joining, 4.4 TB/s of the cache where a copy reaches 4.8; the matrix unit is busy a
// third of the time. 32 sequences of five tokens of 24 heads after 32,769 of 4 x 256, bf16, 4-bit codes
// (shared): 161 us a call among others, 15 of them the joining of 67 MB of partial results (traced,
// each kernel by itself, 158 to 165 and 15); the matrix unit is busy 34 % of the time, the vector unit
// about as much, LDS a quarter; waves wait for LDS operands and at the barrier for the rest.
// Three instances of 32 rows a wave spill: 20 bytes a lane with 256 channels, bf16 q and 4-bit codes, 32
// with 8-bit ones, 12 with 128 channels, fp16 q and 8-bit codes.
#pragma once

#include <math.h>

#include <algorithm>
#include <type_traits>

#include "pn_cache.h"

namespace pn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Division of numbers below 2^31 by a fixed d: n * mul >> shift with mul = floor(2^shift / d) + 1 and
// shift = 31 + ceil(log2 d). (mul * d - 2^shift is at most d <= 2^(shift - 31), so n times it stays
// below 2^shift: exact.) Two instructions for the twenty of a division, in code that runs once and
// cold.
struct FastDiv {
    uint32_t mul;
    int shift;
    FastDiv() = default;
    explicit FastDiv(int d)
    {
        shift = 31;
        while ((int64_t)1 << (shift - 31) < d)
            shift++;
        mul = (uint32_t)(((uint64_t)1 << shift) / (uint32_t)d + 1);
    }
    __device__ __forceinline__ int of(int n) const { return (int)((uint64_t)(uint32_t)n * mul >> shift); }
};

struct AttendArgs {
    CacheView c;
    int type, B, Q, Hq, G;  // G query heads a KV head
    FastDiv by_G, by_Q, by_Hq;
    const void *q;
    int64_t q_seq, q_tok, q_head;
    int q_vec;     // q can be loaded four elements at a time
    float scale;   // of the scores, times log2(e): positive
    float factor;  // of q as it is loaded, for the rest of the scale: its sign, zero, a factor of two
    const int32_t *table, *lens, *q_lens, *prefix_table;
    int64_t table_stride;
    int table_width, prefix_len;
    int prefix_splits, prefix_blocks;  // token ranges and row blocks of the prefix (0 without one)
    int own_splits, own_blocks;        // token ranges of a sequence and row blocks of a KV head
    int shared_tiles;                  // row tiles of a wave in the prefix's shared workgroups, or 0
    int prefix_tiles, own_tiles;       // row tiles of a stream workgroup
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

// Four channels of an output, at a multiple of four.
__device__ __forceinline__ void store4(int type, void *p, int64_t at, f32x4_t x)
{
    typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
    typedef _Float16 f16x4_t __attribute__((ext_vector_type(4)));
    if (type == PN_F32)
        *reinterpret_cast<f32x4_t *>(reinterpret_cast<float *>(p) + at) = x;
    else if (type == PN_BF16)
        *reinterpret_cast<bf16x4_t *>(reinterpret_cast<__bf16 *>(p) + at) = __builtin_convertvector(x, bf16x4_t);
    else
        *reinterpret_cast<f16x4_t *>(reinterpret_cast<_Float16 *>(p) + at) = __builtin_convertvector(x, f16x4_t);
}

// N pieces of eight channels of q, piece i at q + at + 64 (i / 2) + 8 (i % 2), as NT bf16 parts: the value
// rounded, then what that left, and so on: bf16 q has one part, fp16 two, fp32 three, each exact (8, 16
// and 24 bits). A part that more follow stays within bf16's finite numbers, so the largest fp32 numbers
// are made up exactly too, and an infinity is left whole to the last part: rounded to infinity at
// once, either would leave NaN behind. All loads are begun before the first is waited for.
template <int NT, int N>
__device__ __forceinline__ void load_q(const AttendArgs &A, int64_t at, bool live, bf16x8_t (&part)[N][NT])
{
    typedef typename Elem<NT == 1 ? PN_BF16 : NT == 2 ? PN_F16 : PN_F32>::type E;
    typedef E E4 __attribute__((ext_vector_type(4)));
    constexpr float most = 0x1.fep127f;  // bf16's largest
    const E *const p = reinterpret_cast<const E *>(A.q) + (live ? at : 0);
    E4 x[N][2];
    if (A.q_vec) {
#pragma unroll
        for (int i = 0; i < N; i++)
#pragma unroll
            for (int j = 0; j < 2; j++)
                x[i][j] = *reinterpret_cast<const E4 *>(p + 64 * (i / 2) + 8 * (i % 2) + 4 * j);
    } else {
#pragma unroll
        for (int i = 0; i < N; i++)
#pragma unroll
            for (int j = 0; j < 8; j++)
                x[i][j / 4][j % 4] = p[64 * (i / 2) + 8 * (i % 2) + j];
    }
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int j = 0; j < 8; j++) {
            float v = live ? (float)x[i][j / 4][j % 4] * A.factor : 0.0f;
#pragma unroll
            for (int t = 0; t < NT; t++) {
                part[i][t][j] = (__bf16)(t + 1 < NT ? __builtin_amdgcn_fmed3f(v, -most, most) : v);
                v -= (float)part[i][t][j];
            }
        }
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

// The larger of two numbers, the other where one is NaN, up to the largest finite one. (fmaxf would
// first quiet each operand, an instruction apiece.)
__device__ __forceinline__ float larger(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, 0x1.fffffep127f); }

__device__ __forceinline__ float over_groups_max(float v)
{
    float a = v, b = v;
    swap32(a, b);
    v = larger(a, b);
    a = b = v;
    swap16(a, b);
    return larger(a, b);
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

// The scale operand from byte `byte` of an exponent word.
__device__ __forceinline__ float scale_of(uint32_t w, int byte)
{
    return exp_bits(byte == 0 ? w << 23 : byte == 1 ? w << 15 : byte == 2 ? w << 7 : w >> 1);
}

// An offset that is worked out where it is used: beside a uniform base it is one register of the load,
// while the compiler would keep it as a 64-bit one over the whole loop.
__device__ __forceinline__ uint32_t here(uint32_t offset)
{
    asm volatile("" : "+v"(offset));
    return offset;
}

// A lane's part of one 64-channel chunk of a record's K or V, tokens of half a: 16 codes. K: 16 channels
// of a token; V: four channels of four tokens.
template <int FMT>
struct Half {
    static constexpr int N = FMT == PN_CACHE_MXFP8 ? 4 : 2;
    uint32_t d[N];
};
template <int FMT>
struct Chunk {
    Half<FMT> h[2];
};
// Chunk p of the codes at `codes`: 16 bytes a lane and load, a wave's load one contiguous KB (with 8-bit
// codes one a half).
template <int FMT>
__device__ __forceinline__ void load_chunk(const uint8_t *codes, int p, int lane, Chunk<FMT> &c)
{
    const uint32_t at = here(lane * 16);
    if constexpr (FMT == PN_CACHE_MXFP8) {
#pragma unroll
        for (int a = 0; a < 2; a++) {
            const uint4 w = *reinterpret_cast<const uint4 *>(codes + (p * 2 + a) * 1024 + at);
            c.h[a] = Half<FMT>{{w.x, w.y, w.z, w.w}};
        }
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(codes + p * 1024 + at);
        c.h[0] = Half<FMT>{{w.x, w.y}};
        c.h[1] = Half<FMT>{{w.z, w.w}};
    }
}
// Half a of it alone.
template <int FMT>
__device__ __forceinline__ void load_half(const uint8_t *codes, int p, int a, int lane, Half<FMT> &h)
{
    if constexpr (FMT == PN_CACHE_MXFP8) {
        const uint4 w = *reinterpret_cast<const uint4 *>(codes + (p * 2 + a) * 1024 + here(lane * 16));
        h = Half<FMT>{{w.x, w.y, w.z, w.w}};
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(codes + p * 1024 + a * 8 + here(lane * 16));
        h = Half<FMT>{{w.x, w.y}};
    }
}
// Where this lane's exponents are in a record: K's 2 NP bytes [p][a], V's 2 NP words [p][a].
template <int FMT, int D>
__device__ __forceinline__ uint32_t k_exps(int lane)
{
    return here(((lane >> 5) * 16 + (lane & 15)) * Rec<FMT, D>::NP * 2);
}
template <int FMT, int D>
__device__ __forceinline__ uint32_t v_exps(int lane)
{
    return here((((lane >> 3) & 1) * 4 + (lane >> 4)) * Rec<FMT, D>::NP * 8);
}

// K operand: channels 8j .. 8j + 7 of the lane's 16, scale s.
template <int FMT>
__device__ __forceinline__ bf16x8_t k_frag(const Half<FMT> &h, int j, float s)
{
    uint4 r;
    if constexpr (FMT == PN_CACHE_MXFP8)
        r = make_uint4(pair<FMT, 0>(h.d[2 * j], s), pair<FMT, 1>(h.d[2 * j], s),
                       pair<FMT, 0>(h.d[2 * j + 1], s), pair<FMT, 1>(h.d[2 * j + 1], s));
    else
        r = make_uint4(pair<FMT, 0>(h.d[j], s), pair<FMT, 1>(h.d[j], s), pair<FMT, 2>(h.d[j], s),
                       pair<FMT, 3>(h.d[j], s));
    return __builtin_bit_cast(bf16x8_t, r);
}

// V operands of a chunk p: operand n holds channel 64p + 4i + n of the lane's eight tokens; here the
// four of a half, e their exponents.
template <int FMT>
__device__ __forceinline__ void v_half(const Half<FMT> &h, uint32_t e, uint2 (&f)[4])
{
    uint32_t c01[4], c23[4];
#pragma unroll
    for (int t = 0; t < 4; t++) {
        const float s = scale_of(e, t);
        if constexpr (FMT == PN_CACHE_MXFP8) {
            c01[t] = pair<FMT, 0>(h.d[t], s);
            c23[t] = pair<FMT, 1>(h.d[t], s);
        } else if (t & 1) {
            c01[t] = pair<FMT, 2>(h.d[t / 2], s);
            c23[t] = pair<FMT, 3>(h.d[t / 2], s);
        } else {
            c01[t] = pair<FMT, 0>(h.d[t / 2], s);
            c23[t] = pair<FMT, 1>(h.d[t / 2], s);
        }
    }
    constexpr uint32_t lo = 0x05040100, hi = 0x07060302;
    f[0] = make_uint2(__builtin_amdgcn_perm(c01[1], c01[0], lo), __builtin_amdgcn_perm(c01[3], c01[2], lo));
    f[1] = make_uint2(__builtin_amdgcn_perm(c01[1], c01[0], hi), __builtin_amdgcn_perm(c01[3], c01[2], hi));
    f[2] = make_uint2(__builtin_amdgcn_perm(c23[1], c23[0], lo), __builtin_amdgcn_perm(c23[3], c23[2], lo));
    f[3] = make_uint2(__builtin_amdgcn_perm(c23[1], c23[0], hi), __builtin_amdgcn_perm(c23[3], c23[2], hi));
}
template <int FMT>
__device__ __forceinline__ void v_frags(const Chunk<FMT> &v, const uint32_t (&e)[2], bf16x8_t (&f)[4])
{
    uint2 r[2][4];
    v_half<FMT>(v.h[0], e[0], r[0]);
    v_half<FMT>(v.h[1], e[1], r[1]);
#pragma unroll
    for (int n = 0; n < 4; n++)
        f[n] = __builtin_bit_cast(bf16x8_t, make_uint4(r[0][n].x, r[0][n].y, r[1][n].x, r[1][n].y));
}

// Token t of the four in a half of V: zeros.
template <int FMT>
__device__ __forceinline__ void v_clear(Half<FMT> &h, uint32_t &e, int t)
{
    if constexpr (FMT == PN_CACHE_MXFP8)
        h.d[t] = 0;
    else
        h.d[t / 2] &= t & 1 ? 0x0000FFFFu : 0xFFFF0000u;
    e &= ~(255u << (8 * t));
}

// NaN blocks in a record that some rows see only in part: a weight of zero must not meet them. They
// are taken out of V, and what they do to the rows that see them is done here: a product of "is NaN"
// with "is seen" counts, for each row and channel, the NaNs that belong to its sum.
template <int FMT>
__device__ __forceinline__ void v_nan_apart(Chunk<FMT> &v, uint32_t (&e)[2], const f32x4_t (&s)[2],
                                            f32x4_t (&O)[4])
{
    bf16x8_t bad, seen;
#pragma unroll
    for (int a = 0; a < 2; a++)
#pragma unroll
        for (int t = 0; t < 4; t++) {
            const bool nan = ((e[a] >> (8 * t)) & 255u) == 255u;
            bad[4 * a + t] = (__bf16)(nan ? 1.0f : 0.0f);
            seen[4 * a + t] = (__bf16)(s[a][t] == -INFINITY ? 0.0f : 1.0f);
            if (nan)
                v_clear<FMT>(v.h[a], e[a], t);
        }
    const f32x4_t count = mfma(bad, seen, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
    for (int n = 0; n < 4; n++)
#pragma unroll
        for (int r = 0; r < 4; r++)
            O[n][r] = count[r] > 0.0f ? __builtin_nanf("") : O[n][r];
}

// A row's reference m of the weights 2^(s - m) (near its running maximum; all four lanes of a row have
// the same), the lane's own part l of their sum, and O. `base` is -m: infinity before any token.
template <int NP>
struct State {
    float base, l;
    f32x4_t O[NP][4];
    __device__ __forceinline__ void clear()
    {
        base = INFINITY;
        l = 0.0f;
#pragma unroll
        for (int p = 0; p < NP; p++)
#pragma unroll
            for (int n = 0; n < 4; n++)
                O[p][n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
};

// Scores of NR records to weights for RT tiles, as NT bf16 parts in the order of the V operand's tokens.
// The weights are taken against the reference as it is; only where a lane's sum of them passes 2^12
// (or is NaN: no reference yet) are the maximum of its row found, the row's reference moved to it and
// the weights taken again. Weights up to 2^12 lose nothing in fp32 and bf16, and most records need
// neither the maximum, which is as many instructions as the rest, nor a rescaling. The other rows of
// the tile keep their references: a row's roundings do not depend on its neighbours.
template <int NT, int NP, int NR, int RT>
__device__ __forceinline__ void weigh(const f32x4_t (&s)[RT][NR][2], float scale, State<NP> (&st)[RT],
                                      bf16x8_t (&w)[RT][NR][NT])
{
    const auto weights = [&](int rt, float (&x)[NR][8]) {
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < NR; c++) {
#pragma unroll
            for (int a = 0; a < 2; a++)
#pragma unroll
                for (int r = 0; r < 4; r++)
                    x[c][4 * a + r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[rt][c][a][r], scale, st[rt].base));
            const float part = ((x[c][0] + x[c][1]) + (x[c][2] + x[c][3])) + ((x[c][4] + x[c][5]) + (x[c][6] + x[c][7]));
            sum = c ? sum + part : part;
        }
        return sum;
    };
    const auto put = [&](int rt, float (&x)[NR][8]) {
#pragma unroll
        for (int c = 0; c < NR; c++)
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int r = 0; r < 8; r++) {
                    w[rt][c][n][r] = (__bf16)x[c][r];
                    if (n + 1 < NT)
                        x[c][r] -= (float)w[rt][c][n][r];
                }
    };
    float sum[RT];
    bool over = false;
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        float x[NR][8];
        sum[rt] = weights(rt, x);
        over |= !(sum[rt] <= 0x1p12f);
        put(rt, x);
    }
    if (__any(over)) {
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
            float top = -INFINITY;
#pragma unroll
            for (int c = 0; c < NR; c++)
#pragma unroll
                for (int a = 0; a < 2; a++)
                    top = larger(larger(top, larger(s[rt][c][a][0], s[rt][c][a][1])),
                                 larger(s[rt][c][a][2], s[rt][c][a][3]));
            // the rows of lanes i, i + 16, i + 32, i + 48 that are over
            uint64_t rows = __ballot(!(sum[rt] <= 0x1p12f));
            rows |= rows >> 32;
            rows |= rows >> 16;
            top = larger(over_groups_max(top) * scale, -st[rt].base);
            top = (rows >> (threadIdx.x & 15)) & 1 ? top : -st[rt].base;
            // (2^(m - top) of no reference at all: there is nothing to rescale, or it is NaN and stays so)
            const float f = st[rt].base == INFINITY ? 0.0f : __builtin_amdgcn_exp2f(-st[rt].base - top);
            st[rt].l *= f;
#pragma unroll
            for (int p = 0; p < NP; p++)
#pragma unroll
                for (int n = 0; n < 4; n++)
                    st[rt].O[p][n] *= f;
            // no token seen: any finite reference gives weights of zero
            const bool none = top == -INFINITY;
            st[rt].base = none ? 0.0f : -top;
            float x[NR][8];
            sum[rt] = weights(rt, x);
            put(rt, x);
            if (none)
                st[rt].base = INFINITY;
        }
    }
#pragma unroll
    for (int rt = 0; rt < RT; rt++)
        st[rt].l += sum[rt];
}

// Where a row is: its sequence, query token, place in q and in out.
struct Row {
    int b, i;
    int64_t q, out;
};
template <bool OWN>
__device__ __forceinline__ Row row_of(const AttendArgs &A, int b0, int h, int row)
{
    Row r;
    const int qt = A.by_G.of(row);  // query token, counted over all sequences in the prefix
    const int hq = h * A.G + row - qt * A.G;
    r.b = OWN ? b0 : A.by_Q.of(qt);
    r.i = OWN ? qt : qt - r.b * A.Q;
    r.q = r.b * A.q_seq + r.i * A.q_tok + hq * A.q_head;
    r.out = ((int64_t)r.b * A.Q + r.i) * A.Hq + hq;
    return r;
}

// A number that every lane reads and no one writes while the kernel runs, by a scalar load: a vector
// load would be waited for behind the cache's loads in flight.
__device__ __forceinline__ int32_t load_uniform(const int32_t *p)
{
    return *reinterpret_cast<const __attribute__((address_space(4))) int32_t *>(reinterpret_cast<uintptr_t>(p));
}

// Records of KV head h of a sequence's own tokens or of the prefix.
template <int FMT, int D>
struct Records {
    const uint8_t *head;  // the head's first record in page 0
    const int32_t *table;
    int64_t page_bytes;
    int shift, pages;  // log2 of the records a page has; pages of the cache
    __device__ __forceinline__ Records(const AttendArgs &A, const int32_t *table, int h)
        : table(table), shift(A.c.page_shift - 5), pages((int)A.c.pages)
    {
        const int64_t bytes = (int64_t)Rec<FMT, D>::BYTES << shift;  // of one head
        head = A.c.data + h * bytes;
        page_bytes = A.c.heads * bytes;
    }
    __device__ __forceinline__ int page(int t) const { return load_uniform(table + (t >> shift)); }
    // a page number outside the cache is taken as the nearest inside
    __device__ __forceinline__ const uint8_t *at(int page, int t) const
    {
        return head + min(max(page, 0), pages - 1) * page_bytes + (t & ((1 << shift) - 1)) * Rec<FMT, D>::BYTES;
    }
};

constexpr int kWaves = 8;

// A stream workgroup: rows [row0, row0 + 16 tiles) of KV head h over range `split` of a sequence's own
// tokens (OWN) or of the prefix. Wave w has row tile w % tiles and every (8 / tiles)-th record.
// The weights are NW bf16 parts where they meet V: three and two for fp32 and fp16 q, which lose nothing
// that the type keeps, and two for bf16 q as well, so that its output is off by its own rounding alone.
// A second product hides behind the memory here: 4 query tokens of 24 heads over 130,077 of 4 x 256 62.9
// us with one part and 63.3 with two, 16 sequences of 4,096 of 8 x 128 32.2 and 32.3, 32 ragged ones of
// 4 tokens and 96 heads of 64 42.5 and 44.8; the error against 64 bits 2.3e-3 and 1.7e-3, where rounding
// the output makes 1.7e-3.
template <int FMT, int D, int NT, bool OWN>
__device__ __forceinline__ void attend_stream(const AttendArgs &A, int split, int b0, int h, int row0, int tiles,
                                              uint4 *lds)
{
    constexpr int NP = Rec<FMT, D>::NP, NW = NT == 1 ? 2 : NT;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int tile = wave & (tiles - 1), streams = kWaves / tiles, stream = wave / tiles;

    const int nrows = (OWN ? 1 : A.B) * A.Q * A.G;
    const int tokens = OWN ? own_tokens(A, b0) : A.prefix_len;
    const int nq = OWN ? query_tokens(A, b0) : A.Q;
    const int least = OWN ? tokens - nq + 1 : tokens;  // the tokens below are seen by every row
    const Range range = split_range(tokens, OWN ? A.own_splits : A.prefix_splits, split);
    if (range.begin >= range.end && !A.direct)
        return;

    const Records<FMT, D> recs(A, OWN ? A.table + b0 * A.table_stride : A.prefix_table, h);
    Chunk<FMT> kc[NP], vc[NP];
    uint32_t ke[2], ve[NP][2];
    auto load_k = [&](const uint8_t *rec) {
#pragma unroll
        for (int p = 0; p < NP; p++)
            load_chunk<FMT>(rec, p, lane, kc[p]);
        const uint8_t *e = rec + Rec<FMT, D>::KE + k_exps<FMT, D>(lane);
        if constexpr (NP == 1)
            ke[0] = *reinterpret_cast<const uint16_t *>(e);
        else
            ke[0] = *reinterpret_cast<const uint32_t *>(e);
        if constexpr (NP == 4)
            ke[1] = *reinterpret_cast<const uint32_t *>(e + 4);
    };
    auto load_v = [&](const uint8_t *rec) {
        const uint2 *e = reinterpret_cast<const uint2 *>(rec + Rec<FMT, D>::VE + v_exps<FMT, D>(lane));
#pragma unroll
        for (int p = 0; p < NP; p++) {
            load_chunk<FMT>(rec + Rec<FMT, D>::V, p, lane, vc[p]);
            const uint2 t = e[p];
            ve[p][0] = t.x;
            ve[p][1] = t.y;
        }
    };
    int t = range.begin + stream;
    int next_page = 0;
    if (t < range.end) {
        const uint8_t *rec = recs.at(recs.page(t), t);
        load_k(rec);
        load_v(rec);
        if (t + streams < range.end)
            next_page = recs.page(t + streams);
    }

    // q operands to LDS: [tile][p][j][part][lane]
    for (int u = wave; u < tiles * NP; u += kWaves) {
        const int row = row0 + 16 * (u / NP) + i16;
        const Row r = row_of<OWN>(A, b0, h, row < nrows ? row : 0);
        bf16x8_t part[2][NT];
        load_q<NT, 2>(A, r.q + 64 * (u % NP) + 16 * g, row < nrows, part);
#pragma unroll
        for (int n = 0; n < 2 * NT; n++)
            lds[(u * 2 * NT + n) * 64 + lane] = __builtin_bit_cast(uint4, part[n / NT][n % NT]);
    }
    int limit = 0;  // this lane's row sees the tokens below
    {
        const int row = row0 + 16 * tile + i16;
        const Row r = row_of<OWN>(A, b0, h, row < nrows ? row : 0);
        limit = !OWN ? tokens : r.i < nq ? min(tokens, tokens - nq + r.i + 1) : 0;
    }
    __syncthreads();
    const uint4 *const q = lds + tile * NP * 2 * NT * 64 + lane;

    State<NP> state[1];
    State<NP> &st = state[0];
    st.clear();
    for (; t < range.end; t += streams) {
        const bool more = t + streams < range.end;
        const uint8_t *next = recs.at(next_page, t + streams);
        // q stays in LDS: read before the loop, its operands would take the registers of the loads
        // in flight
        int fresh = 0;
        asm volatile("" : "+v"(fresh));

        // q's first parts sum apart from the rest, 2^-8 of them: a third of the roundings at the score's size.
        // One token over 1000, fp32: error against 64 bits 2.9e-7 for 7.1e-7 (four tokens over 130,077
        // 68.1 us for 67.8)
        f32x4_t s[1][1][2] = {{{f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}}}};
        f32x4_t small[2] = {f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}, f32x4_t{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
        for (int p = 0; p < NP; p++)
#pragma unroll
            for (int j = 0; j < 2; j++) {
                bf16x8_t qf[NT];
#pragma unroll
                for (int n = 0; n < NT; n++)
                    qf[n] = __builtin_bit_cast(bf16x8_t, q[((p * 2 + j) * NT + n) * 64 + fresh]);
#pragma unroll
                for (int a = 0; a < 2; a++) {
                    const bf16x8_t kf = k_frag<FMT>(kc[p].h[a], j, scale_of(ke[p >> 1], 2 * (p & 1) + a));
#pragma unroll
                    for (int n = 0; n < NT; n++) {
                        if (n == 0)
                            s[0][0][a] = mfma(kf, qf[n], s[0][0][a]);
                        else
                            small[a] = mfma(kf, qf[n], small[a]);
                    }
                }
            }
        if constexpr (NT > 1) {
#pragma unroll
            for (int a = 0; a < 2; a++)
                s[0][0][a] += small[a];
        }
        if (more) {
            load_k(next);
            if (t + 2 * streams < range.end)
                next_page = recs.page(t + 2 * streams);
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
                    if (first + 16 * a + r >= limit)
                        s[0][0][a][r] = -INFINITY;
                    if (first + 16 * a + r >= tokens) {
#pragma unroll
                        for (int p = 0; p < NP; p++)
                            v_clear<FMT>(vc[p].h[a], ve[p][a], r);
                    }
                }
            if (OWN) {  // a NaN block of a token that only some rows see
                bool any = false;
#pragma unroll
                for (int p = 0; p < NP; p++)
#pragma unroll
                    for (int r = 0; r < 8; r++)
                        any |= ((ve[p][r >> 2] >> (8 * (r & 3))) & 255u) == 255u;
                nan_hidden = __any(any);
            }
        }

        bf16x8_t w[1][1][NW];
        weigh<NW, NP, 1, 1>(s, A.scale, state, w);
        if (nan_hidden) {
#pragma unroll
            for (int p = 0; p < NP; p++)
                v_nan_apart<FMT>(vc[p], ve[p], s[0][0], st.O[p]);
        }
#pragma unroll
        for (int p = 0; p < NP; p++) {
            bf16x8_t vf[4];
            v_frags<FMT>(vc[p], ve[p], vf);
#pragma unroll
            for (int n = 0; n < 4; n++)
#pragma unroll
                for (int e = 0; e < NW; e++)
                    st.O[p][n] = mfma(vf[n], w[0][0][e], st.O[p][n]);
        }
        if (more)
            load_v(next);
    }

    // join the waves of each row tile: O of all waves in LDS, scaled to the tile's common reference,
    // and each wave's part of the sum
    constexpr int PAD = D + 4;
    float *const buf = reinterpret_cast<float *>(lds);  // [wave][row][PAD]
    float *const ms = buf + kWaves * 16 * PAD;          // [wave][row] references, then parts of the sum
    float *const ls = ms + kWaves * 16;
    const float lsum = over_groups_sum(st.l);
    __syncthreads();
    if (g == 0)
        ms[wave * 16 + i16] = -st.base;
    __syncthreads();
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
        const float m = ms[w * 16 + i16];
        top = (w & (tiles - 1)) == tile ? fmaxf(top, m) : top;
    }
    // l = 0 only where a wave saw no token (l is NaN where its scores are)
    const float f = lsum == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(-st.base - top);
#pragma unroll
    for (int p = 0; p < NP; p++)
#pragma unroll
        for (int r = 0; r < 4; r++)
            *reinterpret_cast<f32x4_t *>(buf + (wave * 16 + i16) * PAD + 64 * p + 16 * g + 4 * r) =
                f * f32x4_t{st.O[p][0][r], st.O[p][1][r], st.O[p][2][r], st.O[p][3][r]};
    if (g == 0)
        ls[wave * 16 + i16] = f * lsum;
    __syncthreads();
    const int64_t rows = (int64_t)A.B * A.Q * A.Hq;
    const int64_t slot = (OWN ? A.prefix_splits : 0) + split;
    const auto join = [&](auto tiles_) {
        constexpr int TILES = decltype(tiles_)::value;
#pragma unroll
        for (int u0 = 0; u0 < TILES * 16 * (D / 4); u0 += kWaves * 64) {
            const int u = u0 + threadIdx.x;
            const int cg = u % (D / 4), jr = u / (D / 4) % 16, ti = u / (D / 4) / 16;
            const int row = row0 + 16 * ti + jr;
            if (row >= nrows)
                continue;
            f32x4_t v = {0.0f, 0.0f, 0.0f, 0.0f};
            float sum = 0.0f, most = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWaves; w += TILES) {
                v += *reinterpret_cast<const f32x4_t *>(buf + ((w + ti) * 16 + jr) * PAD + 4 * cg);
                sum += ls[(w + ti) * 16 + jr];
                most = fmaxf(most, ms[(w + ti) * 16 + jr]);
            }
            const Row r = row_of<OWN>(A, b0, h, row);
            const int64_t at = r.out * D + 4 * cg;
            if (A.direct) {
                const bool none = sum == 0.0f || r.i >= nq;  // sees nothing, or not a query token
                store4(A.type, A.out, at, none ? f32x4_t{0.0f, 0.0f, 0.0f, 0.0f} : v * (1.0f / sum));
                if (cg == 0 && A.lse)
                    A.lse[r.out] = none ? -INFINITY : (most + __builtin_amdgcn_logf(sum)) * kLn2;
            } else {
                *reinterpret_cast<f32x4_t *>(A.part + slot * rows * D + at) = v;
                if (cg == 0)
                    A.part_ml[slot * rows + r.out] = make_float2(most, sum);
            }
        }
    };
    if (tiles == 1)
        join(std::integral_constant<int, 1>());
    else if (tiles == 2)
        join(std::integral_constant<int, 2>());
    else
        join(std::integral_constant<int, 4>());
}

// Rows a wave of a shared workgroup can hold at most, in tiles of 16, and the records of a stage: what
// 256 registers take beside the operands in flight (a tile's O takes D / 4, its q D / 8 a part, its
// scores 8 a record, its weights 4 a record and part).
constexpr int shared_tiles(int D, int NT)
{
    return D == 256 ? (NT == 1 ? 2 : 1) : D == 128 ? (NT == 3 ? 1 : 2) : NT == 1 ? 3 : 2;
}
constexpr int stage_records(int D) { return D == 256 ? 1 : 2; }

// Operands read from LDS AHEAD uses early: left to itself the compiler reads two, waits for both and
// starts over, and an LDS read under load takes as long as several uses. begin() starts the first
// reads, run() calls use(i, operand i) for the N operands at `from` (one every 64 uint4). Three ahead,
// also where two would keep 20 bytes a lane less in scratch: 32 sequences of five tokens after 32,769 of
// 4 x 256, bf16, 8-bit codes 170 us with two and 167 with three.
template <int AHEAD>
struct ReadAhead {
    uint4 f[AHEAD];
    __device__ __forceinline__ void begin(const uint4 *from)
    {
#pragma unroll
        for (int i = 0; i < AHEAD; i++)
            f[i] = from[i * 64];
    }
    template <int N, typename F>
    __device__ __forceinline__ void run(const uint4 *from, F use)
    {
#pragma unroll
        for (int i = 0; i < N; i++) {
            use(i, __builtin_bit_cast(bf16x8_t, f[i % AHEAD]));
            if (i + AHEAD < N)
                f[i % AHEAD] = from[(i + AHEAD) * 64];
            __builtin_amdgcn_sched_barrier(0x6);  // (VALU and SALU instructions may move across)
        }
    }
};

// A shared workgroup: rows [row0, row0 + 128 RT) of KV head h over range `split` of the prefix, wave w
// the 16 RT from row0 + 16 RT w. A stage is NR records: K operands [chunk][a][j][lane] in a ring of
// three and V operands [chunk][n][lane] in a ring of two (16 KB each at most). Wave w converts chunk
// w % 4 (64 channels of a record) of K and of V, the tokens of half w / 4.
//
// One barrier a stage: while stage t is used, K of t + 2 and V of t + 1 are written. K(t + 2) takes the
// place of K(t - 1) and V(t + 1) that of V(t - 1), last read before the barrier that ended t - 1; the
// reads of K(t + 1) begin before the barrier that ends t.
// bf16 q's weights meet V rounded to bf16 once (2^-8 at most): a second part costs what the matrix unit
// has least of. 16 sequences after 16,384 of 8 x 128, 8-bit codes 26.0 us with one part and 28.3 with
// two, 32 of five tokens after 32,769 of 4 x 256, 4-bit codes 159 and 215; the error against 64 bits
// 2.4e-3 and 1.7e-3, where rounding the output makes 1.7e-3. (fp32 q takes the same calls without it.)
// (Holding waves 4-7 half a stage behind waves 0-3, so that one wave of a SIMD has the matrix unit while
// the other converts and weighs, took four barriers a stage and came out even.)
template <int FMT, int D, int NT, int RT>
__device__ __forceinline__ void attend_shared(const AttendArgs &A, int split, int h, int row0, uint4 *lds)
{
    constexpr int NP = Rec<FMT, D>::NP, NR = stage_records(D);
    constexpr int STAGE = 1024;  // uint4 of a stage's K or V
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i16 = lane & 15, g = lane >> 4;
    const int nrows = A.B * A.Q * A.G, tokens = A.prefix_len;
    const Range range = split_range(tokens, A.prefix_splits, split);
    if (range.begin >= range.end)
        return;
    const int wrow = row0 + wave * 16 * RT;
    const bool active = wrow < nrows;
    const int limit = min(tokens, range.end * kTile);

    const Records<FMT, D> recs(A, A.prefix_table, h);
    // this wave's half chunk of each stage: chunk cp of the stage's record cr, half a
    const int unit = wave & 3, cr = unit / NP, cp = unit & (NP - 1), a = wave >> 2;
    const bool converts = cr < NR;
    uint4 *const kring = lds, *const vring = lds + 3 * STAGE;
    Half<FMT> kraw, vraw;
    uint32_t ke, ve;
    const uint8_t *krec = nullptr, *vrec = nullptr;  // the records to load next, K a stage ahead of V
    // (records past the range: their place is the last one's, they are loaded and not used)
    auto clamped = [&](int t0) { return min(t0 + cr, range.end - 1); };
    auto load_stage = [&] {
        if (!converts)
            return;
        load_half<FMT>(krec, cp, a, lane, kraw);
        load_half<FMT>(vrec + Rec<FMT, D>::V, cp, a, lane, vraw);
        ke = *reinterpret_cast<const uint8_t *>(krec + Rec<FMT, D>::KE + cp * 2 + a + k_exps<FMT, D>(lane));
        ve = *reinterpret_cast<const uint32_t *>(vrec + Rec<FMT, D>::VE + cp * 8 + a * 4 + v_exps<FMT, D>(lane));
    };
    auto put_k = [&](uint4 *stage) {
        if (!converts)
            return;
#pragma unroll
        for (int j = 0; j < 2; j++)
            stage[(unit * 4 + a * 2 + j) * 64 + lane] =
                __builtin_bit_cast(uint4, k_frag<FMT>(kraw, j, scale_of(ke, 0)));
    };
    auto put_v = [&](int t0, uint4 *stage) {
        if (!converts)
            return;
        if ((t0 + cr + 1) * kTile > limit) {  // past the end: V must not meet a weight of zero as NaN
#pragma unroll
            for (int r = 0; r < 4; r++)
                if ((t0 + cr) * kTile + 16 * a + 4 * g + r >= limit)
                    v_clear<FMT>(vraw, ve, r);
        }
        uint2 f[4];
        v_half<FMT>(vraw, ve, f);
#pragma unroll
        for (int n = 0; n < 4; n++)
            reinterpret_cast<uint2 *>(stage + (unit * 4 + n) * 64 + lane)[a] = f[n];
    };
    const int t_first = range.begin;
    const auto record = [&](int t0) { return recs.at(recs.page(clamped(t0)), clamped(t0)); };
    // the first two stages' loads go out before q's: K and V of the first, K of the second
    krec = vrec = record(t_first);
    load_stage();
    const Half<FMT> k0 = kraw, v0 = vraw;
    const uint32_t ke0 = ke, ve0 = ve;
    krec = vrec = record(t_first + NR);
    load_stage();

    bf16x8_t q[RT][NP * 2][NT];
    State<NP> st[RT];
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        const int row = wrow + 16 * rt + i16;
        const Row r = row_of<false>(A, 0, h, row < nrows ? row : 0);
        load_q<NT, NP * 2>(A, r.q + 16 * g, row < nrows, q[rt]);
        st[rt].clear();
    }
    const Half<FMT> k1 = kraw, v1 = vraw;
    const uint32_t ke1 = ke, ve1 = ve;
    kraw = k0;
    vraw = v0;
    ke = ke0;
    ve = ve0;
    put_k(kring);
    put_v(t_first, vring);
    kraw = k1;
    ke = ke1;
    put_k(kring + STAGE);
    krec = record(t_first + 2 * NR);
    load_stage();  // K of the third stage; V of the second is in hand
    vraw = v1;
    ve = ve1;
    const uint8_t *vnext = krec;
    int page = recs.page(clamped(t_first + 3 * NR));
    ReadAhead<3> ahead;
    __syncthreads();

    int kslot = 0, vslot = 0;  // rings' places of stage t0
    if (active)
        ahead.begin(kring + lane);
    for (int t0 = t_first; t0 < range.end; t0 += NR) {
        const uint4 *const kstage = kring + kslot * STAGE + lane;
        const uint4 *const vstage = vring + vslot * STAGE + lane;
        kslot = kslot == 2 ? 0 : kslot + 1;
        vslot ^= 1;
        vrec = vnext;
        krec = vnext = recs.at(page, clamped(t0 + 3 * NR));
        f32x4_t s[RT][NR][2];
        bf16x8_t w[RT][NR][NT];
        if (active) {
#pragma unroll
            for (int rt = 0; rt < RT; rt++)
#pragma unroll
                for (int c = 0; c < NR; c++)
                    s[rt][c][0] = s[rt][c][1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            ahead.template run<NR * NP * 4>(kstage, [&](int i, bf16x8_t kf) {
                const int c = i / (NP * 4), p = (i >> 2) % NP, b = (i >> 1) & 1, j = i & 1;
#pragma unroll
                for (int rt = 0; rt < RT; rt++)
#pragma unroll
                    for (int n = 0; n < NT; n++)
                        s[rt][c][b] = mfma(kf, q[rt][p * 2 + j][n], s[rt][c][b]);
            });
        }
        page = recs.page(clamped(t0 + 4 * NR));  // here, where no LDS read is waited for with it
        if (active) {
            if ((t0 + NR) * kTile > limit) {
#pragma unroll
                for (int c = 0; c < NR; c++)
#pragma unroll
                    for (int b = 0; b < 2; b++)
#pragma unroll
                        for (int r = 0; r < 4; r++)
                            if ((t0 + c) * kTile + 16 * b + 4 * g + r >= limit) {
#pragma unroll
                                for (int rt = 0; rt < RT; rt++)
                                    s[rt][c][b][r] = -INFINITY;
                            }
            }
            weigh<NT, NP, NR, RT>(s, A.scale, st, w);
            __builtin_amdgcn_sched_barrier(0);  // (the scores' registers are free by now)
            ahead.begin(vstage);
            ahead.template run<NR * NP * 4>(vstage, [&](int i, bf16x8_t vf) {
                const int c = i / (NP * 4), p = (i >> 2) % NP, n = i & 3;
#pragma unroll
                for (int rt = 0; rt < RT; rt++)
#pragma unroll
                    for (int e = 0; e < NT; e++)
                        st[rt].O[p][n] = mfma(vf, w[rt][c][e], st[rt].O[p][n]);
            });
            ahead.begin(kring + kslot * STAGE + lane);
        }
        put_k(kring + (kslot == 2 ? 0 : kslot + 1) * STAGE);
        put_v(t0 + NR, vring + vslot * STAGE);
        load_stage();
        __syncthreads();
    }

    const int64_t rows = (int64_t)A.B * A.Q * A.Hq;
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        const int row = wrow + 16 * rt + i16;
        const float lsum = over_groups_sum(st[rt].l);
        if (row < nrows) {
            const Row r = row_of<false>(A, 0, h, row);
            float *const to = A.part + (split * rows + r.out) * D + 16 * g;
#pragma unroll
            for (int p = 0; p < NP; p++)
#pragma unroll
                for (int e = 0; e < 4; e++)
                    *reinterpret_cast<f32x4_t *>(to + 64 * p + 4 * e) = f32x4_t{
                        st[rt].O[p][0][e], st[rt].O[p][1][e], st[rt].O[p][2][e], st[rt].O[p][3][e]};
            if (g == 0)
                A.part_ml[split * rows + r.out] = make_float2(-st[rt].base, lsum);
        }
    }
}

// Workgroups: first the prefix's [row block][range][KV head], so that the row blocks that read the
// same tokens run on one XCD where their number allows, then the own tokens' [range][sequence][row
// block][KV head]. RT: tiles of 16 rows a wave holds in the prefix's shared workgroups (0: they are
// stream workgroups, if any).
// Stream workgroups of up to 128 channels keep within 128 registers, so that two are on a CU where the
// call has that many: 100 sequences of four tokens over 10 to 1000 of 8 x 128, fp32 39.4 us, and 49.3
// with the 129 registers that the compiler takes by itself.
template <int FMT, int D, int NT, int RT>
__global__ void __launch_bounds__(512, RT == 0 && D <= 128 ? 4 : 2) attend_kernel(AttendArgs A)
{
    extern __shared__ uint4 lds[];
    int id = blockIdx.x;
    const int each = A.c.heads * A.prefix_splits;
    if (id < each * A.prefix_blocks) {
        const int block = id / each, rest = id - block * each;
        const int split = rest / A.c.heads, h = rest - split * A.c.heads;
        if constexpr (RT > 0)
            attend_shared<FMT, D, NT, RT>(A, split, h, block * 128 * RT, lds);
        else
            attend_stream<FMT, D, NT, false>(A, split, 0, h, block * 16 * A.prefix_tiles, A.prefix_tiles, lds);
        return;
    }
    id -= each * A.prefix_blocks;
    const int h = id % A.c.heads;
    id /= A.c.heads;
    const int block = id % A.own_blocks;
    id /= A.own_blocks;
    const int b = id % A.B;
    attend_stream<FMT, D, NT, true>(A, id / A.B, b, h, block * 16 * A.own_tiles, A.own_tiles, lds);
}

// The ranges that a row has results of: `n`, the first `np` of the prefix.
struct Live {
    int np, n, prefix_splits;
    __device__ __forceinline__ Live(const AttendArgs &A, int64_t row) : prefix_splits(A.prefix_splits)
    {
        const int qt = A.by_Hq.of((int)row), b = A.by_Q.of(qt), i = qt - b * A.Q;
        np = A.prefix_splits ? live_ranges(A.prefix_len, A.prefix_splits) : 0;
        n = np + live_ranges(own_tokens(A, b), A.own_splits);
        if (i >= query_tokens(A, b))
            n = np = 0;
    }
    __device__ __forceinline__ int64_t slot(int k) const { return k < np ? k : prefix_splits + k - np; }
};

// Few rows: joins the ranges of 64 channels of a row in a workgroup, thread = four channels of every
// 16th range. Bound by its start and two dependent loads: 96 rows of 256 channels and 64 ranges 4.8 us.
template <int D>
__global__ void __launch_bounds__(256) attend_join_kernel(AttendArgs A)
{
    constexpr int NP = D / 64;
    constexpr int AHEAD = 4;  // ranges a thread has in flight
    __shared__ f32x4_t part[16][16];
    __shared__ float sums[16];
    const int lane = threadIdx.x & 63, cg = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int64_t rows = (int64_t)A.B * A.Q * A.Hq;
    const int64_t row = blockIdx.x / NP;
    const int p = blockIdx.x - (int)row * NP;
    const Live live(A, row);
    const int n = live.n;
    const auto slot = [&](int k) { return live.slot(k); };
    f32x4_t o[AHEAD];
    float2 ml[AHEAD];
    const auto load = [&](int k0) {
#pragma unroll
        for (int k = 0; k < AHEAD; k++) {
            const int r = k0 + 16 * k;
            ml[k] = r < n ? A.part_ml[slot(r) * rows + row] : make_float2(0.0f, 0.0f);
            o[k] = r < n ? *reinterpret_cast<const f32x4_t *>(A.part + (slot(r) * rows + row) * D + 64 * p + 4 * cg)
                         : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        }
    };
    load(rg);
    float top = -INFINITY;  // every wave finds the maximum by itself
    for (int k = lane; k < n; k += 64)
        top = fmaxf(top, A.part_ml[slot(k) * rows + row].x);
#pragma unroll
    for (int s = 32; s > 0; s >>= 1)
        top = fmaxf(top, __shfl_xor(top, s, 64));
    float sum = 0.0f;
    f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = rg; k0 < n; k0 += 16 * AHEAD) {
        if (k0 > rg)
            load(k0);
#pragma unroll
        for (int k = 0; k < AHEAD; k++)
            if (ml[k].y != 0.0f) {
                const float f = __builtin_amdgcn_exp2f(ml[k].x - top);
                sum += f * ml[k].y;
                acc += f * o[k];
            }
    }
    part[rg][cg] = acc;
    if (cg == 0)
        sums[rg] = sum;
    __syncthreads();
    if (rg != 0)
        return;
    sum = 0.0f;
    acc = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < 16; r++) {
        sum += sums[r];
        acc += part[r][cg];
    }
    const bool none = sum == 0.0f;
    const float inv = 1.0f / sum;
    store4(A.type, A.out, row * D + 64 * p + 4 * cg, none ? f32x4_t{0.0f, 0.0f, 0.0f, 0.0f} : acc * inv);
    if (p == 0 && cg == 0 && A.lse)
        A.lse[row] = none ? -INFINITY : (top + __builtin_amdgcn_logf(sum)) * kLn2;
}

// Many rows: a wave joins 256 / D rows, D / 4 lanes a row, eight ranges in flight. 3,840 rows of 256
// channels and 18 ranges: 15 us, 4.7 TB/s.
template <int D>
__global__ void __launch_bounds__(256) attend_join_rows_kernel(AttendArgs A)
{
    constexpr int L = D / 4;  // lanes a row
    const int64_t rows = (int64_t)A.B * A.Q * A.Hq;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t row = at / L;
    const int cg = (int)(at % L);
    if (row >= rows)
        return;
    const Live live(A, row);
    float m = -INFINITY, sum = 0.0f;
    f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = 0; k0 < live.n; k0 += 8) {  // eight ranges in flight
        float2 ml[8];
        f32x4_t o[8];
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const int64_t i = live.slot(min(k0 + k, live.n - 1)) * rows + row;
            ml[k] = A.part_ml[i];
            o[k] = *reinterpret_cast<const f32x4_t *>(A.part + i * D + 4 * cg);
            if (k0 + k >= live.n)
                ml[k] = make_float2(-INFINITY, 0.0f);
        }
        float top = m;
#pragma unroll
        for (int k = 0; k < 8; k++)
            top = fmaxf(top, ml[k].x);
        const float f0 = sum == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m - top);
        m = top;
        sum *= f0;
        acc *= f0;
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (ml[k].y != 0.0f) {
                const float f = __builtin_amdgcn_exp2f(ml[k].x - m);
                sum += f * ml[k].y;
                acc += f * o[k];
            }
    }
    const bool none = sum == 0.0f;
    const float inv = 1.0f / sum;
    store4(A.type, A.out, row * D + 4 * cg, none ? f32x4_t{0.0f, 0.0f, 0.0f, 0.0f} : acc * inv);
    if (cg == 0 && A.lse)
        A.lse[row] = none ? -INFINITY : (m + __builtin_amdgcn_logf(sum)) * kLn2;
}

template <int FMT, int D, int NT, int RT>
static int launch_attend(const AttendArgs &A, hipStream_t s)
{
    constexpr auto kern = attend_kernel<FMT, D, NT, RT>;
    // q operands of a stream workgroup, the joining of its waves, or a shared one's rings (3 of K, 2 of V)
    const int tiles = std::max(A.own_tiles, RT > 0 ? 1 : A.prefix_tiles);
    const int bytes = std::max(std::max(tiles * (D / 32) * NT * 1024, kWaves * 16 * (D + 4 + 2) * 4), RT > 0 ? 5 * 16384 : 0);
    if (!lds_limit_once<kern>(160 * 1024))
        return PN_ERR_HIP;
    const int64_t rows = (int64_t)A.B * A.Q * A.Hq;
    const int64_t grid = (int64_t)A.c.heads * A.prefix_splits * A.prefix_blocks +
                         (int64_t)A.own_splits * A.B * A.own_blocks * A.c.heads;
    hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(kWaves * 64), bytes, s, A);
    const int st = launch_status();
    if (st != PN_OK || A.direct)
        return st;
    // D / 4 lanes a row where the rows alone fill the CUs with a wave each: 3,840 rows of 256 channels,
    // 18 ranges 29 us a workgroup a row, 15 so; below, the workgroups a row have more loads in flight
    if (rows >= 1024)
        hipLaunchKernelGGL((attend_join_rows_kernel<D>), dim3((unsigned)((rows * (D / 4) + 255) / 256)),
                           dim3(256), 0, s, A);
    else
        hipLaunchKernelGGL((attend_join_kernel<D>), dim3((unsigned)(rows * (D / 64))), dim3(256), 0, s, A);
    return launch_status();
}

template <int FMT, int D, int NT>
static int launch_tiles(const AttendArgs &A, hipStream_t s)
{
    constexpr int MOST = shared_tiles(D, NT);
    if (A.shared_tiles == 0)
        return launch_attend<FMT, D, NT, 0>(A, s);
    if (A.shared_tiles == 1)
        return launch_attend<FMT, D, NT, 1>(A, s);
    if (MOST >= 2 && A.shared_tiles == 2)
        return launch_attend<FMT, D, NT, MOST >= 2 ? 2 : 1>(A, s);
    return launch_attend<FMT, D, NT, MOST>(A, s);
}

// Launches format FMT, one source file each. parts: of q (1, 2, 3).
template <int FMT>
int launch_format(const AttendArgs &A, int dim, int parts, hipStream_t s);

#define PN_ATTEND_DIM(FMT, D)                                                                      \
    return parts == 1   ? launch_tiles<FMT, D, 1>(A, s)                                            \
           : parts == 2 ? launch_tiles<FMT, D, 2>(A, s)                                            \
                        : launch_tiles<FMT, D, 3>(A, s);
#define PN_ATTEND_FORMAT(FMT)                                                                      \
    template <>                                                                                    \
    int launch_format<FMT>(const AttendArgs &A, int dim, int parts, hipStream_t s)                 \
    {                                                                                              \
        if (dim == 64) {                                                                           \
            PN_ATTEND_DIM(FMT, 64)                                                                 \
        } else if (dim == 128) {                                                                   \
            PN_ATTEND_DIM(FMT, 128)                                                                \
        }                                                                                          \
        PN_ATTEND_DIM(FMT, 256)                                                                    \
    }

}  // namespace pn
