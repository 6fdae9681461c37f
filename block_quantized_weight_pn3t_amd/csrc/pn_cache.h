// pn_cache.h -- the microscaled key/value cache on the device: where the codes and exponent bytes of
// a token lie (the layout that pn.h states), and plain element types.
#pragma once

#include "pn_common.h"

namespace pn {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

constexpr int kTile = 32;  // tokens a record

// Sizes and offsets of a record for FMT and D channels: K codes at 0, V codes, K and V exponents.
template <int FMT, int D>
struct Rec {
    static constexpr int NP = D / 64;                                    // chunks of 64 channels
    static constexpr int CODES = FMT == PN_CACHE_MXFP8 ? kTile * D : kTile * D / 2;
    static constexpr int V = CODES, KE = 2 * CODES, VE = KE + D, BYTES = VE + D;
};

inline int rec_bytes(int format, int dim) { return (format == PN_CACHE_MXFP8 ? 66 : 34) * dim; }

struct CacheView {
    uint8_t *data;
    int64_t pages;
    int heads;
    int page_shift;  // log2 of the tokens a page has
};

// PN_OK and the view, or the first thing that is wrong with the cache's description.
int cache_view(const pn_cache *c, CacheView &view);

// Bytes of one element of a plain type, 0 if unknown.
inline int elem_bytes(int type)
{
    return type == PN_F32 ? 4 : type == PN_BF16 || type == PN_F16 ? 2 : 0;
}

template <int T> struct Elem;
template <> struct Elem<PN_F32> { typedef float type; };
template <> struct Elem<PN_BF16> { typedef __bf16 type; };
template <> struct Elem<PN_F16> { typedef _Float16 type; };

// v in fp32, for good: left to itself the compiler rounds a double that ends in 16 bits to them directly,
// which takes up to thirty instructions.
__device__ __forceinline__ float to_f32(double v)
{
    float f = (float)v;
    asm("" : "+v"(f));
    return f;
}

}  // namespace pn
