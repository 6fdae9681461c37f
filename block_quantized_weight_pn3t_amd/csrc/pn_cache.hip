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
#include "pn_cache_put.h"

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
            put_k<FMT, D>(krec, kp, p, ku, kx[i][p]);
            put_v<FMT, D>(vrec, vp, p, vu, vx[i][p]);
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
    if (T < 0 || !tokens_fit(T, c.heads, kQuads * 4))
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
    if (T < 0 || !tokens_fit(T, c.heads, 16))
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
