// pn_cache.hip -- keys and values quantised into the microscaled cache, and read back, on gfx950.
//
// A block of 32 channels x with largest magnitude A: exponent byte b, the smallest (>= 16) with
// A <= M * 2^(b - 127), M = 448 (E4M3) or 6 (E2M1); codes rne(x * 2^(127 - b)). The byte comes from
// the bits of A: its exponent field minus log2 of M's binade (8 or 2), plus one where A's mantissa
// passes M's (1.75 or 1.5). x * 2^(127 - b) is exact (a power of two), so a code is rounded once.
//
// Both directions move each number once and do almost no arithmetic: memory bound. A workgroup takes
// consecutive tokens of one KV head, a wave four of them (writing 32, a wave four twice; reading 16):
// neighbouring tokens share cache lines of the record, and workgroups run on different XCDs, each with
// its own cache. Measured: 16,384 tokens of 4 x 256 bf16 written in 26 us (3.9 TB/s; 33 with the heads of
// four tokens in a workgroup); 32,768 read in 34 us (6.0 TB/s; 52.5 so, and with cached stores).
//
// In V, a code dword is four channels of one token and four tokens' dwords are neighbours, so lane =
// token + 4 * channel group: where the four tokens have consecutive slots (the usual run) a store covers
// whole 256-byte runs of the record. In K, 16 channels of one token are 16 contiguous bytes and
// neighbouring tokens' pieces are neighbours: lane = 4-channel group of the piece + 4 * token + 16 *
// piece.
#include "pn_cache.h"

namespace pn {

int cache_view(const pn_cache *c, CacheView &view)
{
    if (!c)
        return PN_ERR_NULL;
    if (c->format != PN_CACHE_MXFP8 && c->format != PN_CACHE_MXFP4)
        return PN_ERR_FORMAT;
    if (pn_cache_page_bytes(c->format, c->heads, c->dim, c->page) == 0 || c->pages < 0 ||
        c->pages > INT32_MAX)
        return PN_ERR_SHAPE;
    if (c->pages > 0 && !c->data)
        return PN_ERR_NULL;
    if (!aligned(c->data, 16))
        return PN_ERR_ALIGN;
    view = CacheView{(uint8_t *)c->data, c->pages, c->heads, __builtin_ctz((unsigned)c->page)};
    return PN_OK;
}

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

constexpr int kQuads = 8;  // groups of four tokens a workgroup takes

struct Plain {  // a plain tensor of keys or values, strides in elements
    const void *p;
    int64_t token, head;
};

template <int FMT, int D, int T, bool VEC>
__global__ void __launch_bounds__(256) cache_write_kernel(CacheView c, Plain k, Plain v,
                                                          const int64_t *__restrict__ slots,
                                                          int64_t ntok)
{
    constexpr int NP = Rec<FMT, D>::NP;
    const int lane = threadIdx.x & 63;
    const uint32_t run = blockIdx.x / (uint32_t)c.heads;
    const int h = (int)(blockIdx.x - run * (uint32_t)c.heads);
    // K: lane = e + 4 * token + 16 * g; V: lane = token + 4 * u
    const int kt = (lane >> 2) & 3, ku = (lane & 3) + 4 * (lane >> 4);
    const int vt = lane & 3, vu = lane >> 2;
    const int64_t first = ((int64_t)run * kQuads + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * 4;
    f32x4_t kx[2][NP], vx[2][NP];
    int64_t kslot[2], vslot[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const int64_t kat = first + 16 * i + kt, vat = first + 16 * i + vt;
        const int64_t ktok = min(kat, ntok - 1), vtok = min(vat, ntok - 1);
        kslot[i] = kat < ntok ? slots[ktok] : -1;
        vslot[i] = vat < ntok ? slots[vtok] : -1;
#pragma unroll
        for (int p = 0; p < NP; p++) {
            kx[i][p] = load4<T, VEC>(k.p, ktok * k.token + h * k.head + 64 * p + 4 * ku);
            vx[i][p] = load4<T, VEC>(v.p, vtok * v.token + h * v.head + 64 * p + 4 * vu);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; i++) {
        if (first + 16 * i >= ntok)
            break;
        uint8_t *const krec = record_of<FMT, D>(c, kslot[i], h);
        uint8_t *const vrec = record_of<FMT, D>(c, vslot[i], h);
        const int kp = (int)(kslot[i] & 31), vp = (int)(vslot[i] & 31);
#pragma unroll
        for (int p = 0; p < NP; p++) {
            // a K block is lanes that differ in bits 0, 1 and 4; a V block in bits 2, 3 and 4
            const int kb = exponent_byte<FMT>(block_top<false>(kx[i][p]));
            const int vb = exponent_byte<FMT>(block_top<true>(vx[i][p]));
            const uint32_t kw = encode4<FMT>(kx[i][p], kb), vw = encode4<FMT>(vx[i][p], vb);
            if (krec) {
                uint8_t *const at = krec + k_code_at<FMT, D>(kp, p, ku);
                if constexpr (FMT == PN_CACHE_MXFP8)
                    *reinterpret_cast<uint32_t *>(at) = kw;
                else
                    *reinterpret_cast<uint16_t *>(at) = (uint16_t)kw;
                if ((ku & 7) == 0)
                    krec[k_exp_at<FMT, D>(kp, p, ku >> 3)] = (uint8_t)kb;
            }
            if (vrec) {
                uint8_t *const at = vrec + v_code_at<FMT, D>(vp, p, vu);
                if constexpr (FMT == PN_CACHE_MXFP8)
                    *reinterpret_cast<uint32_t *>(at) = vw;
                else
                    *reinterpret_cast<uint16_t *>(at) = (uint16_t)vw;
                if ((vu & 7) == 0)
                    vrec[v_exp_at<FMT, D>(vp, p, vu >> 3)] = (uint8_t)vb;
            }
        }
    }
}

// Four codes as fp32 numbers: the conversion to bf16 applies 2^(b - 127) exactly (NaN at 255).
template <int FMT>
__device__ __forceinline__ f32x4_t decode4(uint32_t w, uint32_t b)
{
    const float s = __builtin_bit_cast(float, b << 23);
    bf16x2_t lo, hi;
    if constexpr (FMT == PN_CACHE_MXFP8) {
        lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false);
        hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true);
    } else {
        lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
        hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    }
    return f32x4_t{(float)lo.x, (float)lo.y, (float)hi.x, (float)hi.y};
}

template <int T>
__device__ __forceinline__ void store4(void *base, int64_t at, f32x4_t x)
{
    typedef typename Elem<T>::type E;
    typedef E E4 __attribute__((ext_vector_type(4)));
    // past the caches: kept there, the output would push out the lines that neighbouring waves share
    __builtin_nontemporal_store(E4{(E)x[0], (E)x[1], (E)x[2], (E)x[3]},
                                reinterpret_cast<E4 *>(reinterpret_cast<E *>(base) + at));
}

template <int FMT, int D, int T>
__global__ void __launch_bounds__(256) cache_read_kernel(CacheView c,
                                                         const int64_t *__restrict__ slots,
                                                         int64_t ntok, void *__restrict__ k,
                                                         void *__restrict__ v)
{
    constexpr int NP = Rec<FMT, D>::NP;
    const int lane = threadIdx.x & 63;
    const uint32_t run = blockIdx.x / (uint32_t)c.heads;
    const int h = (int)(blockIdx.x - run * (uint32_t)c.heads);
    const int64_t quad = (int64_t)run * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (quad * 4 >= ntok)
        return;
    const int kt = (lane >> 2) & 3, ku = (lane & 3) + 4 * (lane >> 4);
    const int vt = lane & 3, vu = lane >> 2;
    const int64_t ktok = quad * 4 + kt, vtok = quad * 4 + vt;
    const int64_t kslot = ktok < ntok ? slots[ktok] : -1;
    const int64_t vslot = vtok < ntok ? slots[vtok] : -1;
    const uint8_t *const krec = record_of<FMT, D>(c, kslot, h);
    const uint8_t *const vrec = record_of<FMT, D>(c, vslot, h);
    const int kp = (int)(kslot & 31), vp = (int)(vslot & 31);
    uint32_t kw[NP], vw[NP], kb[NP], vb[NP];
#pragma unroll
    for (int p = 0; p < NP; p++) {
        kw[p] = vw[p] = kb[p] = vb[p] = 0;
        if (krec) {
            const uint8_t *const at = krec + k_code_at<FMT, D>(kp, p, ku);
            kw[p] = FMT == PN_CACHE_MXFP8 ? *reinterpret_cast<const uint32_t *>(at)
                                          : *reinterpret_cast<const uint16_t *>(at);
            kb[p] = krec[k_exp_at<FMT, D>(kp, p, ku >> 3)];
        }
        if (vrec) {
            const uint8_t *const at = vrec + v_code_at<FMT, D>(vp, p, vu);
            vw[p] = FMT == PN_CACHE_MXFP8 ? *reinterpret_cast<const uint32_t *>(at)
                                          : *reinterpret_cast<const uint16_t *>(at);
            vb[p] = vrec[v_exp_at<FMT, D>(vp, p, vu >> 3)];
        }
    }
#pragma unroll
    for (int p = 0; p < NP; p++) {
        if (ktok < ntok)
            store4<T>(k, (ktok * c.heads + h) * D + 64 * p + 4 * ku, decode4<FMT>(kw[p], kb[p]));
        if (vtok < ntok)
            store4<T>(v, (vtok * c.heads + h) * D + 64 * p + 4 * vu, decode4<FMT>(vw[p], vb[p]));
    }
}

template <int FMT, int D, int T>
static int launch_write(const CacheView &c, Plain k, Plain v, bool vec, const int64_t *slots,
                        int64_t ntok, hipStream_t s)
{
    const dim3 grid((unsigned)((ntok + kQuads * 4 - 1) / (kQuads * 4) * c.heads));
    if (vec)
        hipLaunchKernelGGL((cache_write_kernel<FMT, D, T, true>), grid, dim3(256), 0, s, c, k, v,
                           slots, ntok);
    else
        hipLaunchKernelGGL((cache_write_kernel<FMT, D, T, false>), grid, dim3(256), 0, s, c, k, v,
                           slots, ntok);
    return launch_status();
}

template <int FMT, int D, int T>
static int launch_read(const CacheView &c, const int64_t *slots, int64_t ntok, void *k, void *v,
                       hipStream_t s)
{
    const dim3 grid((unsigned)((ntok + 15) / 16 * c.heads));
    hipLaunchKernelGGL((cache_read_kernel<FMT, D, T>), grid, dim3(256), 0, s, c, slots, ntok, k, v);
    return launch_status();
}

// Calls F::template go<FMT, D, T>() for the run-time format, dim and type (all checked before).
template <typename F>
static int by_kind(int fmt, int dim, int type, F f)
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

struct WriteCall {
    CacheView c;
    Plain k, v;
    bool vec;
    const int64_t *slots;
    int64_t ntok;
    hipStream_t s;
    template <int FMT, int D, int T>
    int operator()()
    {
        return launch_write<FMT, D, T>(c, k, v, vec, slots, ntok, s);
    }
};

struct ReadCall {
    CacheView c;
    const int64_t *slots;
    int64_t ntok;
    void *k, *v;
    hipStream_t s;
    template <int FMT, int D, int T>
    int operator()()
    {
        return launch_read<FMT, D, T>(c, slots, ntok, k, v, s);
    }
};

// Tokens of one call: its token quads and heads are counted in 32 bits.
static bool tokens_fit(int64_t ntok, int heads)
{
    return ntok <= (int64_t)1 << 40 && (ntok + 3) / 4 * heads < INT32_MAX;
}

}  // namespace pn

using namespace pn;

extern "C" int64_t pn_cache_page_bytes(int format, int heads, int dim, int page)
{
    if ((format != PN_CACHE_MXFP8 && format != PN_CACHE_MXFP4) || heads < 1 || heads > 65536 ||
        (dim != 64 && dim != 128 && dim != 256) || page < 32 || page > 1024 || (page & (page - 1)))
        return 0;
    return (int64_t)heads * (page / kTile) * rec_bytes(format, dim);
}

extern "C" int pn_cache_write(const pn_cache *cache, int type, const void *k, int64_t k_token_stride,
                              int64_t k_head_stride, const void *v, int64_t v_token_stride,
                              int64_t v_head_stride, const int64_t *slots, int64_t T, void *stream)
{
    CacheView c;
    int st = cache_view(cache, c);
    if (st != PN_OK)
        return st;
    const int size = elem_bytes(type);
    if (size == 0)
        return PN_ERR_FORMAT;
    if (T < 0 || !tokens_fit(T, c.heads))
        return PN_ERR_SHAPE;
    if (T == 0)
        return PN_OK;
    if (!k || !v || !slots)
        return PN_ERR_NULL;
    if (!aligned(k, size) || !aligned(v, size) || !aligned(slots, 8))
        return PN_ERR_ALIGN;
    if ((st = check_device()) != PN_OK)
        return st;
    const bool vec = aligned(k, 4 * size) && aligned(v, 4 * size) &&
                     ((k_token_stride | k_head_stride | v_token_stride | v_head_stride) & 3) == 0;
    return by_kind(cache->format, cache->dim, type,
                   WriteCall{c, Plain{k, k_token_stride, k_head_stride},
                             Plain{v, v_token_stride, v_head_stride}, vec, slots, T,
                             (hipStream_t)stream});
}

extern "C" int pn_cache_read(const pn_cache *cache, int type, const int64_t *slots, int64_t T,
                             void *k, void *v, void *stream)
{
    CacheView c;
    int st = cache_view(cache, c);
    if (st != PN_OK)
        return st;
    const int size = elem_bytes(type);
    if (size == 0)
        return PN_ERR_FORMAT;
    if (T < 0 || !tokens_fit(T, c.heads))
        return PN_ERR_SHAPE;
    if (T == 0)
        return PN_OK;
    if (!k || !v || !slots)
        return PN_ERR_NULL;
    if (!aligned(k, 4 * size) || !aligned(v, 4 * size) || !aligned(slots, 8))
        return PN_ERR_ALIGN;
    if ((st = check_device()) != PN_OK)
        return st;
    return by_kind(cache->format, cache->dim, type,
                   ReadCall{c, slots, T, k, v, (hipStream_t)stream});
}
