// pn_cache_put.h -- what writes the microscaled cache share: numbers to codes and an exponent byte, and
// where they go.
#pragma once

#include "pn_cache.h"
#include "pn_launch.h"

namespace pn {

constexpr int kQuads = 8;  // groups of four tokens a workgroup takes

struct Plain {  // a plain tensor of keys or values, strides in elements
    const void *p;
    int64_t token, head;
};

// Four consecutive elements as fp32; one load where they are aligned to 4 elements (VEC).
template <int T, bool VEC>
__device__ __forceinline__ f32x4_t load4(const void *base, int64_t at)
{
    typedef typename Elem<T>::type E;
    typedef E E4 __attribute__((ext_vector_type(4)));
    const E *p = reinterpret_cast<const E *>(base) + at;
    if constexpr (VEC) {
        const E4 v = *reinterpret_cast<const E4 *>(p);
        return f32x4_t{(float)v.x, (float)v.y, (float)v.z, (float)v.w};
    } else {
        return f32x4_t{(float)p[0], (float)p[1], (float)p[2], (float)p[3]};
    }
}

// The larger of v and v moved within each row of 16 lanes.
template <int CTRL>
__device__ __forceinline__ uint32_t larger_of(uint32_t v)
{
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true));
}

// The largest magnitude's bits of a block of 8 lanes: those that differ in the lane bits 0, 1 and 4 (K)
// or 2, 3 and 4 (V).
template <bool V>
__device__ __forceinline__ uint32_t block_top(f32x4_t x)
{
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float f = x[j];
        m = max(m, __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu);
    }
    if constexpr (V)
        m = larger_of<0x128>(larger_of<0x124>(m));  // row_ror 4, then 8
    else
        m = larger_of<0x4E>(larger_of<0xB1>(m));  // quad_perm [1,0,3,2], then [2,3,0,1]
    const auto p = __builtin_amdgcn_permlane16_swap(m, m, false, false);
    return max((uint32_t)p[0], (uint32_t)p[1]);
}

template <int FMT>
__device__ __forceinline__ int exponent_byte(uint32_t top)
{
    constexpr int emax = FMT == PN_CACHE_MXFP8 ? 8 : 2;
    constexpr uint32_t most = FMT == PN_CACHE_MXFP8 ? 0x600000u : 0x400000u;
    const int e = (int)(top >> 23);
    return e >= 254 ? 255 : max(e - emax + ((top & 0x7FFFFFu) > most ? 1 : 0), 16);
}

// The codes of four numbers with exponent byte b, in the low 32 (8-bit) or 16 (4-bit) bits. Nothing
// saturates: the block's largest is within the type by the choice of b.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(f32x4_t x, int b)
{
    if (b == 255)
        return 0;
    // 2^(127 - b): b is 16..253, the power 2^111..2^-126
    const float up = __builtin_bit_cast(float, (uint32_t)(254 - b) << 23);
    if constexpr (FMT == PN_CACHE_MXFP8) {
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(x[0] * up, x[1] * up, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(x[2] * up, x[3] * up, w, true);
        return (uint32_t)w;
    } else {
        uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0] * up, x[1] * up, 1.0f, 0);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2] * up, x[3] * up, 1.0f, 1);
        return w & 0xFFFFu;
    }
}

// Offsets inside a record. `tok` is the token's place in the record (0..31), u the 4-channel group
// of the 64-channel chunk p.
template <int FMT, int D>
__device__ __forceinline__ int k_code_at(int tok, int p, int u)
{
    const int a = tok >> 4, i = tok & 15, g = u >> 2, e = u & 3;
    return FMT == PN_CACHE_MXFP8 ? ((((p * 2 + a) * 4 + g) * 16 + i) * 4 + e) * 4
                                 : ((((p * 4 + g) * 16 + i) * 2 + a) * 4 + e) * 2;
}
template <int FMT, int D>
__device__ __forceinline__ int v_code_at(int tok, int p, int u)
{
    const int a = tok >> 4, g = (tok >> 2) & 3, t = tok & 3;
    return Rec<FMT, D>::V + (FMT == PN_CACHE_MXFP8 ? ((((p * 2 + a) * 4 + g) * 16 + u) * 4 + t) * 4
                                                   : ((((p * 4 + g) * 16 + u) * 2 + a) * 4 + t) * 2);
}
template <int FMT, int D>
__device__ __forceinline__ int k_exp_at(int tok, int p, int half)
{
    return Rec<FMT, D>::KE + ((half * 16 + (tok & 15)) * Rec<FMT, D>::NP + p) * 2 + (tok >> 4);
}
template <int FMT, int D>
__device__ __forceinline__ int v_exp_at(int tok, int p, int half)
{
    return Rec<FMT, D>::VE +
           (((half * 4 + ((tok >> 2) & 3)) * Rec<FMT, D>::NP + p) * 2 + (tok >> 4)) * 4 + (tok & 3);
}

// The record that holds slot, head h; nullptr where the slot is not in the cache.
template <int FMT, int D>
__device__ __forceinline__ uint8_t *record_of(const CacheView &c, int64_t slot, int h)
{
    if (slot < 0 || (slot >> c.page_shift) >= c.pages)
        return nullptr;
    const int64_t page = slot >> c.page_shift;
    const int tile = (int)(slot & ((1 << c.page_shift) - 1)) / kTile;
    return c.data + (((page * c.heads + h) << (c.page_shift - 5)) + tile) * Rec<FMT, D>::BYTES;
}

// Four channels x of a token's key, group u of chunk p: code and exponent into the record at its place
// `tok` (nowhere where there is no record). A block is the lanes that differ in bits 0, 1 and 4.
template <int FMT, int D>
__device__ __forceinline__ void put_k(uint8_t *rec, int tok, int p, int u, f32x4_t x)
{
    const int b = exponent_byte<FMT>(block_top<false>(x));
    const uint32_t w = encode4<FMT>(x, b);
    if (rec) {
        uint8_t *const at = rec + k_code_at<FMT, D>(tok, p, u);
        if constexpr (FMT == PN_CACHE_MXFP8)
            *reinterpret_cast<uint32_t *>(at) = w;
        else
            *reinterpret_cast<uint16_t *>(at) = (uint16_t)w;
        if ((u & 7) == 0)
            rec[k_exp_at<FMT, D>(tok, p, u >> 3)] = (uint8_t)b;
    }
}
// The same of a value: lanes that differ in bits 2, 3 and 4.
template <int FMT, int D>
__device__ __forceinline__ void put_v(uint8_t *rec, int tok, int p, int u, f32x4_t x)
{
    const int b = exponent_byte<FMT>(block_top<true>(x));
    const uint32_t w = encode4<FMT>(x, b);
    if (rec) {
        uint8_t *const at = rec + v_code_at<FMT, D>(tok, p, u);
        if constexpr (FMT == PN_CACHE_MXFP8)
            *reinterpret_cast<uint32_t *>(at) = w;
        else
            *reinterpret_cast<uint16_t *>(at) = (uint16_t)w;
        if ((u & 7) == 0)
            rec[v_exp_at<FMT, D>(tok, p, u >> 3)] = (uint8_t)b;
    }
}

// Calls F::template go<FMT, D, T>() for the run-time format, dim and type (all checked before).
template <typename F>
inline int by_kind(int fmt, int dim, int type, F f)
{
#define PN_KIND(FMT, D)                                                                            \
    if (fmt == FMT && dim == D)                                                                    \
        return type == PN_F32    ? f.template operator()<FMT, D, PN_F32>()                         \
               : type == PN_BF16 ? f.template operator()<FMT, D, PN_BF16>()                        \
                                 : f.template operator()<FMT, D, PN_F16>();
    PN_KIND(PN_CACHE_MXFP8, 64)
    PN_KIND(PN_CACHE_MXFP8, 128)
    PN_KIND(PN_CACHE_MXFP8, 256)
    PN_KIND(PN_CACHE_MXFP4, 64)
    PN_KIND(PN_CACHE_MXFP4, 128)
    PN_KIND(PN_CACHE_MXFP4, 256)
#undef PN_KIND
    return PN_ERR_SHAPE;
}

// Tokens of one call, `each` of them and a head a workgroup of 256 threads: what one launch takes.
inline bool tokens_fit(int64_t ntok, int heads, int each)
{
    return ntok <= (int64_t)1 << 40 && (ntok + each - 1) / each * heads <= launch_most(256);
}

}  // namespace pn
