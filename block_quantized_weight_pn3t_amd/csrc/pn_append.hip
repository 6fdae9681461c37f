// pn_append.hip -- queries and keys rotated by their tokens' positions, keys and values into the
// microscaled cache, on gfx950.
//
// A pair of channels (a, b) turns to (a cos - b sin, a sin + b cos), cosine and sine from the token's row of
// a table. Products of fp32 numbers are exact in 64 bits, so a rotated number is the exact one rounded at
// 2^-53 and once to fp32: a key's codes and exponents are fixed by the definition, whatever the order in
// which this computes.
//
// Memory bound: every query, key and value is read once and written once. One launch, two kinds of
// workgroup:
//   cache    32 tokens of one KV head, dealt to the lanes as pn_cache_write deals them. A key's lane holds
//            four channels and loads its partner's four beside them (the same cache lines, so no more
//            memory traffic).
//   queries  a thread has a token, both halves of four or eight pairs (or as many channels that stay) and some
//            heads, so cosines and sines are loaded once for all of them and queries once.
//
// Measured: 16,384 tokens of 24 and 4 heads of 256, bf16, all channels turned 111 us (4.7 TB/s; a copy reaches
// 4.9); 8192 of them in fp32, a quarter turned, 98 us (5.0); with four heads a thread and eight channels 134 us, too
// few waves; with channels that stay in a branch of their own 79 us for 52 of bf16, a quarter turned; queries
// kept in the caches as they are written, 3 % more.
#include <algorithm>

#include "pn_cache_put.h"

namespace pn {

// Heads a thread of the queries' workgroups turns, with `channels` a unit (as many as leave room for four waves a SIMD).
__host__ __device__ constexpr int turn_heads(int channels, bool pairs) { return channels == 8 && !pairs ? 2 : 4; }

struct AppendArgs {
    Plain k, v, q;
    int64_t q_out_token, q_out_head;
    void *q_out;
    const float *rotation;
    const int64_t *positions, *slots;
    int64_t rows, T;
    int rot, Hq, cache_blocks;  // workgroups of the first kind, before the others
    int units;         // of a token and head
    int units_mul;     // n / units = n * units_mul >> 16 for n < 256
    int tokens_a_block, head_blocks;
};

__device__ __forceinline__ const float *table_row(const AppendArgs &A, int64_t token)
{
    const int64_t at = A.positions ? A.positions[token] : token;
    return A.rotation + min(max(at, (int64_t)0), A.rows - 1) * A.rot;
}

// a c - b s and a s + b c.
__device__ __forceinline__ float turn_a(float a, float b, float c, float s)
{
    return to_f32(__builtin_fma((double)a, (double)c, -((double)b * (double)s)));
}
__device__ __forceinline__ float turn_b(float a, float b, float c, float s)
{
    return to_f32(__builtin_fma((double)a, (double)s, (double)b * (double)c));
}

// Two pairs of neighbouring channels.
__device__ __forceinline__ f32x4_t turn_pairs(f32x4_t x, f32x2_t c, f32x2_t s)
{
    return f32x4_t{turn_a(x[0], x[1], c[0], s[0]), turn_b(x[0], x[1], c[0], s[0]),
                   turn_a(x[2], x[3], c[1], s[1]), turn_b(x[2], x[3], c[1], s[1])};
}

// CH channels of a query: 16 bytes where they are aligned (VEC), one by one elsewhere. What goes out is read by the
// next kernel at the earliest, so it is not kept in the caches that the rest passes through.
template <int T, int CH, bool VEC>
__device__ __forceinline__ void get(const void *base, int64_t at, float (&x)[CH])
{
    typedef typename Elem<T>::type E;
    typedef E EV __attribute__((ext_vector_type(CH)));
    const E *const p = reinterpret_cast<const E *>(base) + at;
    if constexpr (VEC) {
        const EV v = *reinterpret_cast<const EV *>(p);
#pragma unroll
        for (int j = 0; j < CH; j++)
            x[j] = (float)v[j];
    } else {
#pragma unroll
        for (int j = 0; j < CH; j++)
            x[j] = (float)p[j];
    }
}
template <int T, int CH, bool VEC>
__device__ __forceinline__ void put(void *base, int64_t at, const float (&x)[CH])
{
    typedef typename Elem<T>::type E;
    typedef E EV __attribute__((ext_vector_type(CH)));
    E *const p = reinterpret_cast<E *>(base) + at;
    if constexpr (VEC) {
        EV v;
#pragma unroll
        for (int j = 0; j < CH; j++)
            v[j] = (E)x[j];
        __builtin_nontemporal_store(v, reinterpret_cast<EV *>(p));
    } else {
#pragma unroll
        for (int j = 0; j < CH; j++)
            p[j] = (E)x[j];
    }
}
// CH cosines or sines.
template <int CH>
__device__ __forceinline__ void get_angles(const float *p, float (&x)[CH])
{
#pragma unroll
    for (int i = 0; i < CH; i += CH % 4 ? 2 : 4)
        if constexpr (CH % 4) {
            const f32x2_t v = *reinterpret_cast<const f32x2_t *>(p + i);
            x[i] = v[0];
            x[i + 1] = v[1];
        } else {
            const f32x4_t v = *reinterpret_cast<const f32x4_t *>(p + i);
#pragma unroll
            for (int j = 0; j < 4; j++)
                x[i + j] = v[j];
        }
}

// Keys and values of 32 tokens of a KV head.
template <int FMT, int D, int T, bool VEC, bool PAIRS>
__device__ __forceinline__ void append_cache(const CacheView &c, const AppendArgs &A, uint32_t block)
{
    constexpr int NP = Rec<FMT, D>::NP;
    const int lane = threadIdx.x & 63;
    const uint32_t run = block / (uint32_t)c.heads;
    const int h = (int)(block - run * (uint32_t)c.heads);
    const int kt = (lane >> 2) & 3, ku = (lane & 3) + 4 * (lane >> 4);
    const int vt = lane & 3, vu = lane >> 2;
    const int64_t first = ((int64_t)run * kQuads + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 4;
    const int half = A.rot / 2;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        if (first + 16 * i >= A.T)
            break;
        const int64_t kat = first + 16 * i + kt, vat = first + 16 * i + vt;
        const int64_t ktok = min(kat, A.T - 1), vtok = min(vat, A.T - 1);
        const int64_t kslot = kat < A.T ? A.slots[ktok] : -1, vslot = vat < A.T ? A.slots[vtok] : -1;
        const float *const row = table_row(A, ktok);
        const int64_t kbase = ktok * A.k.token + h * A.k.head;
        f32x4_t kx[NP], vx[NP];
#pragma unroll
        for (int p = 0; p < NP; p++) {
            const int ch = 64 * p + 4 * ku;
            kx[p] = load4<T, VEC>(A.k.p, kbase + ch);
            vx[p] = load4<T, VEC>(A.v.p, vtok * A.v.token + h * A.v.head + 64 * p + 4 * vu);
        }
#pragma unroll
        for (int p = 0; p < NP; p++) {
            const int ch = 64 * p + 4 * ku;
            if (ch < A.rot) {
                if constexpr (PAIRS) {
                    kx[p] = turn_pairs(kx[p], *reinterpret_cast<const f32x2_t *>(row + ch / 2),
                                       *reinterpret_cast<const f32x2_t *>(row + half + ch / 2));
                } else {
                    const bool a = ch < half;
                    const int j = a ? ch : ch - half;
                    const f32x4_t other = load4<T, VEC>(A.k.p, kbase + (a ? ch + half : j));
                    const f32x4_t cs = *reinterpret_cast<const f32x4_t *>(row + j);
                    const f32x4_t sn = *reinterpret_cast<const f32x4_t *>(row + half + j);
                    // a: a cos - b sin; b: b cos + a sin
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        kx[p][e] = turn_a(kx[p][e], other[e], cs[e], a ? sn[e] : -sn[e]);
                }
            }
        }
        uint8_t *const krec = record_of<FMT, D>(c, kslot, h);
        uint8_t *const vrec = record_of<FMT, D>(c, vslot, h);
#pragma unroll
        for (int p = 0; p < NP; p++) {
            put_k<FMT, D>(krec, (int)(kslot & 31), p, ku, kx[p]);
            put_v<FMT, D>(vrec, (int)(vslot & 31), p, vu, vx[p]);
        }
    }
}

// Queries of some tokens and kTurn heads, CH channels a unit.
template <int T, int CH, bool VEC, bool PAIRS>
__device__ __forceinline__ void turn_queries(const AppendArgs &A, uint32_t block)
{
    constexpr int kTurn = turn_heads(CH, PAIRS);
    const uint32_t run = block / (uint32_t)A.head_blocks;
    const int h0 = (int)(block - run * (uint32_t)A.head_blocks) * kTurn;
    const int n = ((int)threadIdx.x * A.units_mul) >> 16;
    const int u = (int)threadIdx.x - n * A.units;
    const int64_t token = (int64_t)run * A.tokens_a_block + n;
    if (n >= A.tokens_a_block || token >= A.T)
        return;
    const int heads = min(kTurn, A.Hq - h0), half = A.rot / 2;
    const int64_t from = token * A.q.token + h0 * A.q.head, to = token * A.q_out_token + h0 * A.q_out_head;
    const int turned = A.rot / (PAIRS ? CH : 2 * CH);  // units that turn
    const bool turns = u < turned;
    if constexpr (PAIRS) {
        // CH channels: pairs of neighbours, or they stay
        const int ch = CH * u;
        float x[kTurn][CH];
#pragma unroll
        for (int i = 0; i < kTurn; i++)
            if (i < heads)
                get<T, CH, VEC>(A.q.p, from + i * A.q.head + ch, x[i]);
        if (turns) {
            const float *const row = table_row(A, token) + ch / 2;
            float c[CH / 2], s[CH / 2];
            get_angles<CH / 2>(row, c);
            get_angles<CH / 2>(row + half, s);
#pragma unroll
            for (int i = 0; i < kTurn; i++)
                if (i < heads)
#pragma unroll
                    for (int j = 0; j < CH / 2; j++) {
                        const float a = x[i][2 * j], b = x[i][2 * j + 1];
                        x[i][2 * j] = turn_a(a, b, c[j], s[j]);
                        x[i][2 * j + 1] = turn_b(a, b, c[j], s[j]);
                    }
        }
#pragma unroll
        for (int i = 0; i < kTurn; i++)
            if (i < heads)
                put<T, CH, VEC>(A.q_out, to + i * A.q_out_head + ch, x[i]);
    } else {
        // twice CH channels: both halves of pairs, or neighbours that stay
        const int ch = turns ? CH * u : A.rot + 2 * CH * (u - turned), other = ch + (turns ? half : CH);
        float a[kTurn][CH], b[kTurn][CH];
#pragma unroll
        for (int i = 0; i < kTurn; i++)
            if (i < heads) {
                get<T, CH, VEC>(A.q.p, from + i * A.q.head + ch, a[i]);
                get<T, CH, VEC>(A.q.p, from + i * A.q.head + other, b[i]);
            }
        if (turns) {
            const float *const row = table_row(A, token) + ch;
            float c[CH], s[CH];
            get_angles<CH>(row, c);
            get_angles<CH>(row + half, s);
#pragma unroll
            for (int i = 0; i < kTurn; i++)
                if (i < heads)
#pragma unroll
                    for (int e = 0; e < CH; e++) {
                        const float x = a[i][e], y = b[i][e];
                        a[i][e] = turn_a(x, y, c[e], s[e]);
                        b[i][e] = turn_b(x, y, c[e], s[e]);
                    }
        }
#pragma unroll
        for (int i = 0; i < kTurn; i++)
            if (i < heads) {
                put<T, CH, VEC>(A.q_out, to + i * A.q_out_head + ch, a[i]);
                put<T, CH, VEC>(A.q_out, to + i * A.q_out_head + other, b[i]);
            }
    }
}

// CH: channels of a query's unit, VEC of q and q_out (and, with fewer channels, of k and v) aligned to it.
template <int FMT, int D, int T, int CH, bool VEC, bool PAIRS>
__global__ void __launch_bounds__(256) append_kernel(CacheView c, AppendArgs A)
{
    if (blockIdx.x < (uint32_t)A.cache_blocks)
        append_cache<FMT, D, T, VEC, PAIRS>(c, A, blockIdx.x);
    else
        turn_queries<T, CH, VEC, PAIRS>(A, blockIdx.x - (uint32_t)A.cache_blocks);
}

struct AppendCall {
    CacheView c;
    AppendArgs A;
    int channels;  // of a query's unit: 8 or 4
    bool vec, pairs;
    uint32_t blocks;
    hipStream_t s;
    template <int FMT, int D, int T, int CH, bool VEC>
    int launch()
    {
        if (pairs)
            hipLaunchKernelGGL((append_kernel<FMT, D, T, CH, VEC, true>), dim3(blocks), dim3(256), 0, s, c, A);
        else
            hipLaunchKernelGGL((append_kernel<FMT, D, T, CH, VEC, false>), dim3(blocks), dim3(256), 0, s, c, A);
        return launch_status();
    }
    template <int FMT, int D, int T>
    int operator()()
    {
        if constexpr (T != PN_F32)
            if (channels == 8)
                return launch<FMT, D, T, 8, true>();
        return vec ? launch<FMT, D, T, 4, true>() : launch<FMT, D, T, 4, false>();
    }
};

}  // namespace pn

using namespace pn;

extern "C" int pn_cache_append(const pn_cache *cache, const pn_append_args *a, void *stream)
{
    CacheView c;
    int st = cache_view(cache, c);
    if (st != PN_OK)
        return st;
    if (!a)
        return PN_ERR_NULL;
    const int size = elem_bytes(a->type);
    if (size == 0)
        return PN_ERR_FORMAT;
    if (a->T < 0 || !tokens_fit(a->T, c.heads, kQuads * 4) || a->rows < 1 || a->rot < 8 || a->rot % 8 || a->rot > cache->dim ||
        (a->interleaved != 0 && a->interleaved != 1) || (!a->positions && a->rows < a->T) || (a->q && a->Hq < 1))
        return PN_ERR_SHAPE;
    if (a->T == 0)
        return PN_OK;
    if (!a->k || !a->v || !a->slots || !a->rotation || (a->q && !a->q_out))
        return PN_ERR_NULL;
    if (!aligned(a->k, size) || !aligned(a->v, size) || !aligned(a->q, size) || !aligned(a->q_out, size) ||
        !aligned(a->slots, 8) || !aligned(a->positions, 8) || !aligned(a->rotation, 16))
        return PN_ERR_ALIGN;
    AppendArgs A = {};
    A.k = Plain{a->k, a->k_token_stride, a->k_head_stride};
    A.v = Plain{a->v, a->v_token_stride, a->v_head_stride};
    A.rotation = a->rotation;
    A.positions = a->positions;
    A.slots = a->slots;
    A.rows = a->rows;
    A.T = a->T;
    A.rot = a->rot;
    int64_t strides = A.k.token | A.k.head | A.v.token | A.v.head;
    int64_t blocks = (a->T + kQuads * 4 - 1) / (kQuads * 4) * c.heads;
    A.cache_blocks = (int)blocks;
    bool vec = aligned(a->k, 4 * size) && aligned(a->v, 4 * size);
    int channels = 4;
    if (a->q) {
        A.q = Plain{a->q, a->q_token_stride, a->q_head_stride};
        A.q_out = a->q_out;
        A.q_out_token = a->q_out_token_stride;
        A.q_out_head = a->q_out_head_stride;
        A.Hq = a->Hq;
        strides |= A.q.token | A.q.head | A.q_out_token | A.q_out_head;
        vec = vec && aligned(a->q, 4 * size) && aligned(a->q_out, 4 * size) && (strides & 3) == 0;
        // eight channels of 16 bits are a load of 16 bytes
        if (size == 2 && vec && aligned(a->q, 16) && aligned(a->q_out, 16) &&
            ((A.q.token | A.q.head | A.q_out_token | A.q_out_head) & 7) == 0 && a->rot % (a->interleaved ? 8 : 16) == 0)
            channels = 8;
        // channels that stay are left alone where the queries are turned in place
        const bool in_place = a->q == a->q_out && a->q_token_stride == a->q_out_token_stride &&
                              a->q_head_stride == a->q_out_head_stride;
        A.units = (in_place ? a->rot : cache->dim) / (a->interleaved ? channels : 2 * channels);
        A.units_mul = (65536 + A.units - 1) / A.units;
        A.tokens_a_block = 256 / A.units;
        const int turn = turn_heads(channels, a->interleaved);
        A.head_blocks = (A.Hq - 1) / turn + 1;
        const int64_t runs = (a->T + A.tokens_a_block - 1) / A.tokens_a_block;
        if (runs > INT32_MAX / A.head_blocks)
            return PN_ERR_SHAPE;
        blocks += runs * A.head_blocks;
    }
    if (blocks > launch_most(256))
        return PN_ERR_SHAPE;
    if ((st = check_device()) != PN_OK)
        return st;
    return by_kind(cache->format, cache->dim, a->type,
                   AppendCall{c, A, channels, vec && (strides & 3) == 0, a->interleaved != 0, (uint32_t)blocks,
                              (hipStream_t)stream});
}
