// pn_norm.hip -- the residual's addition, the root-mean-square norm and 8-bit rows, on gfx950.
//
// h = x + residual (rounded to its type), y = h r w, r = 1 / sqrt(mean h^2 + eps). An 8-bit row of
// t = h w has codes rint(127 t / T), T = max |t|; r is the same for all of a row, so it leaves the codes
// alone and T and the sum of squares come out of one pass.
//
// Memory bound: every number is read once, held in registers while the row's sum and maximum are made,
// and written once. One workgroup a row, or one wave where the row fits it: no barrier, four rows a
// workgroup.
//
// Products h w are exact in 64 bits. A code is computed in fp32, where it is off by less than 1e-4, and in
// 64 bits, by the definition, where it lies that near to a border (two numbers in ten thousand).
#include <float.h>

#include "pn_cache.h"

namespace pn {

struct NormArgs {
    int64_t rows, x_stride, residual_stride, sum_stride, out_stride;
    int K;
    const void *x, *residual, *weight;
    void *sum, *out;
    int8_t *codes;
    float *scales;
    int weight_type;
    float eps;
};


// N elements at p[at], one load of 16 bytes for each eight (two for fp32).
template <int T, int N>
__device__ __forceinline__ void load_n(const void *p, int64_t at, float (&x)[N])
{
    typedef typename Elem<T>::type E;
    typedef E EN __attribute__((ext_vector_type(N), aligned(N == 1 ? sizeof(E) : 16)));
    const EN v = *reinterpret_cast<const EN *>(reinterpret_cast<const E *>(p) + at);
#pragma unroll
    for (int j = 0; j < N; j++)
        x[j] = (float)v[j];
}
template <int T, int N>
__device__ __forceinline__ void store_n(void *p, int64_t at, const float (&x)[N])
{
    typedef typename Elem<T>::type E;
    typedef E EN __attribute__((ext_vector_type(N), aligned(N == 1 ? sizeof(E) : 16)));
    EN v;
#pragma unroll
    for (int j = 0; j < N; j++)
        v[j] = (E)x[j];
    *reinterpret_cast<EN *>(reinterpret_cast<E *>(p) + at) = v;
}

// The weights of a thread's N elements, of any type.
template <int N>
__device__ __forceinline__ void load_weight(int type, const void *p, int at, float (&w)[N])
{
    if (type == PN_F32)
        load_n<PN_F32, N>(p, at, w);
    else if (type == PN_BF16)
        load_n<PN_BF16, N>(p, at, w);
    else
        load_n<PN_F16, N>(p, at, w);
}

__device__ __forceinline__ double wave_sum64(double v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v += __shfl_xor(v, o, 64);
    return v;
}
__device__ __forceinline__ double wave_max64(double v)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v = fmax(v, __shfl_xor(v, o, 64));
    return v;
}

// rint((127 t) / T): `t` and `inv` = 127 / T in fp32 where that is enough, `exact` gives t in 64 bits.
template <typename F>
__device__ __forceinline__ int code_of(float t, float inv, bool plain, double T, F exact)
{
    const float c = t * inv, n = rintf(c);
    int code = (int)n;
    if (!plain || !(fabsf(c - n) < 0.4999f))
        code = (int)rint((127.0 * exact()) / T);
    return code;
}

// NORM: the norm with a weight; else the numbers' 8-bit rows alone. VEC: elements a load (8, or 1 for rows
// that are not aligned). NV: pieces of VEC elements a thread holds. WAVE: a wave a row.
template <int T, bool NORM, int VEC, int NV, bool WAVE>
__global__ void __launch_bounds__(1024) norm_kernel(NormArgs A)
{
    __shared__ double lds[2][16];
    __shared__ int lds_bad[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int threads = WAVE ? 64 : (int)blockDim.x, thread = WAVE ? lane : (int)threadIdx.x;
    const int64_t row = WAVE ? (int64_t)blockIdx.x * (blockDim.x >> 6) + wave : (int64_t)blockIdx.x;
    if (WAVE && row >= A.rows)
        return;

    float h[NV][VEC];
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int at = (i * threads + thread) * VEC;
        if (at < A.K)
            load_n<T, VEC>(A.x, row * A.x_stride + at, h[i]);
    }
    if (NORM && A.residual) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int at = (i * threads + thread) * VEC;
            if (at < A.K) {
                float r[VEC];
                load_n<T, VEC>(A.residual, row * A.residual_stride + at, r);
#pragma unroll
                for (int j = 0; j < VEC; j++)
                    h[i][j] = (float)(typename Elem<T>::type)(h[i][j] + r[j]);
            }
        }
    }
    // the weights stay in registers where there is room, else they are read again (from the caches)
    constexpr bool HOLD = NV * VEC <= 32;
    float held[HOLD ? NV : 1][VEC];
    double top = 0.0;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int at = (i * threads + thread) * VEC;
        if (at >= A.K)
            continue;
        float (&w)[VEC] = held[HOLD ? i : 0];
        if constexpr (NORM) {
            if (A.sum)
                store_n<T, VEC>(A.sum, row * A.sum_stride + at, h[i]);
            load_weight<VEC>(A.weight_type, A.weight, at, w);
        }
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            if constexpr (NORM) {
                const double d = (double)h[i][j];
                ss = fma(d, d, ss);
                top = fmax(top, fabs(d * (double)w[j]));
                bad |= !(fabsf(w[j]) <= FLT_MAX);
            } else {
                top = fmax(top, (double)fabsf(h[i][j]));
            }
            bad |= !(fabsf(h[i][j]) <= FLT_MAX);
        }
    }
    top = wave_max64(top);
    if constexpr (NORM)
        ss = wave_sum64(ss);
    int any = __any(bad);
    if constexpr (!WAVE) {
        if (lane == 0) {
            lds[0][wave] = top;
            lds[1][wave] = ss;
            lds_bad[wave] = any;
        }
        __syncthreads();
        top = ss = 0.0;
        any = 0;
        for (int v = 0; v < (int)blockDim.x >> 6; v++) {
            top = fmax(top, lds[0][v]);
            ss += lds[1][v];
            any |= lds_bad[v];
        }
    }
    const double r = NORM ? 1.0 / sqrt(ss / A.K + (double)A.eps) : 1.0;
    const bool none = any || !(r < INFINITY);  // no finite numbers in the row
    const float inv = (float)(127.0 / top);
    const bool plain = top > 0x1p-100 && top < 0x1p100;
    if (A.scales && thread == 0)
        A.scales[row] = none ? __builtin_nanf("") : (float)(top * r / 127.0);
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int at = (i * threads + thread) * VEC;
        if (at >= A.K)
            continue;
        float (&w)[VEC] = held[HOLD ? i : 0];
        if constexpr (NORM) {
            if (!HOLD)
                load_weight<VEC>(A.weight_type, A.weight, at, w);
            if (A.out) {
                float y[VEC];
#pragma unroll
                for (int j = 0; j < VEC; j++)
                    y[j] = to_f32((double)h[i][j] * r * (double)w[j]);
                store_n<T, VEC>(A.out, row * A.out_stride + at, y);
            }
        }
        if (A.codes) {
            int c[VEC];
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                const float t = NORM ? h[i][j] * w[j] : h[i][j];
                c[j] = none || !(top > 0.0) ? 0 : code_of(t, inv, plain, top, [&] {
                    return NORM ? (double)h[i][j] * (double)w[j] : (double)h[i][j];
                });
            }
            int8_t *const p = A.codes + row * A.K + at;
            if constexpr (VEC == 8) {
                uint2 b = make_uint2(0, 0);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    b.x |= ((uint32_t)c[j] & 255u) << (8 * j);
                    b.y |= ((uint32_t)c[4 + j] & 255u) << (8 * j);
                }
                *reinterpret_cast<uint2 *>(p) = b;
            } else {
                *p = (int8_t)c[0];
            }
        }
    }
}

template <int T, bool NORM, int VEC, int NV, bool WAVE>
static void launch_norm(const NormArgs &A, int threads, hipStream_t s)
{
    const int per = WAVE ? 4 : 1;
    hipLaunchKernelGGL((norm_kernel<T, NORM, VEC, NV, WAVE>), dim3((unsigned)((A.rows + per - 1) / per)),
                       dim3(WAVE ? 256 : threads), 0, s, A);
}

template <int T, bool NORM>
static int run_norm(const NormArgs &A, bool vec, hipStream_t s)
{
    const auto wide = [](int pieces, int nv) { return ((pieces + nv - 1) / nv + 63) / 64 * 64; };
    if (vec) {
        const int pieces = A.K / 8;
        if (pieces <= 64)
            launch_norm<T, NORM, 8, 1, true>(A, 0, s);
        else if (pieces <= 128)
            launch_norm<T, NORM, 8, 2, true>(A, 0, s);
        else if (pieces <= 512)
            launch_norm<T, NORM, 8, 1, false>(A, wide(pieces, 1), s);
        else if (pieces <= 1024)
            launch_norm<T, NORM, 8, 2, false>(A, wide(pieces, 2), s);
        else if (pieces <= 4096)
            launch_norm<T, NORM, 8, 4, false>(A, wide(pieces, 4), s);
        else
            launch_norm<T, NORM, 8, 8, false>(A, wide(pieces, 8), s);
    } else {
        if (A.K <= 512)
            launch_norm<T, NORM, 1, 8, true>(A, 0, s);
        else if (A.K <= 8192)
            launch_norm<T, NORM, 1, 8, false>(A, wide(A.K, 8), s);
        else
            launch_norm<T, NORM, 1, 64, false>(A, wide(A.K, 64), s);
    }
    return launch_status();
}

template <bool NORM>
static int by_type(int type, const NormArgs &A, bool vec, hipStream_t s)
{
    return type == PN_F32    ? run_norm<PN_F32, NORM>(A, vec, s)
           : type == PN_BF16 ? run_norm<PN_BF16, NORM>(A, vec, s)
                             : run_norm<PN_F16, NORM>(A, vec, s);
}

// Rows and widths that the kernels take.
static bool rows_fit(int64_t rows, int64_t K)
{
    return rows >= 0 && rows <= INT32_MAX && K >= 1 && K <= PN_ROW_MAX_WIDTH;
}

// Whether rows of `size`-byte elements at p take loads of eight elements (16-byte pieces).
static bool eights(const void *p, int64_t stride, int size) { return aligned(p, 16) && (stride * size & 15) == 0; }

}  // namespace pn

using namespace pn;

extern "C" int pn_int8_quantize_rows(int type, const void *x, int64_t x_stride, int64_t N, int64_t K,
                                     int8_t *codes, float *scales, void *stream)
{
    const int size = elem_bytes(type);
    if (size == 0)
        return PN_ERR_FORMAT;
    if (!rows_fit(N, K))
        return PN_ERR_SHAPE;
    if (N == 0)
        return PN_OK;
    if (!x || !codes || !scales)
        return PN_ERR_NULL;
    if (!aligned(x, size) || !aligned(scales, 4))
        return PN_ERR_ALIGN;
    const int st = check_device();
    if (st != PN_OK)
        return st;
    NormArgs A = {};
    A.rows = N;
    A.K = (int)K;
    A.x = x;
    A.x_stride = x_stride;
    A.codes = codes;
    A.scales = scales;
    return by_type<false>(type, A, K % 8 == 0 && eights(x, x_stride, size) && aligned(codes, 8), (hipStream_t)stream);
}

extern "C" int pn_add_norm(const pn_add_norm_args *a, void *stream)
{
    if (!a)
        return PN_ERR_NULL;
    const int size = elem_bytes(a->type), wsize = elem_bytes(a->weight_type);
    if (size == 0 || wsize == 0)
        return PN_ERR_FORMAT;
    if (!rows_fit(a->rows, a->K) || !(a->eps >= 0.0f && a->eps <= FLT_MAX))
        return PN_ERR_SHAPE;
    if (a->rows == 0)
        return PN_OK;
    if (!a->x || !a->weight || (!a->out && !a->codes) || !a->codes != !a->scales)
        return PN_ERR_NULL;
    if (!aligned(a->x, size) || !aligned(a->residual, size) || !aligned(a->sum, size) || !aligned(a->out, size) ||
        !aligned(a->weight, wsize) || !aligned(a->scales, 4))
        return PN_ERR_ALIGN;
    const int st = check_device();
    if (st != PN_OK)
        return st;
    const NormArgs A{a->rows, a->x_stride, a->residual_stride, a->sum_stride, a->out_stride, (int)a->K,
                     a->x, a->residual, a->weight, a->sum, a->out, a->codes, a->scales, a->weight_type, a->eps};
    const bool vec = a->K % 8 == 0 && eights(a->x, a->x_stride, size) &&
                     (!a->residual || eights(a->residual, a->residual_stride, size)) &&
                     (!a->sum || eights(a->sum, a->sum_stride, size)) &&
                     (!a->out || eights(a->out, a->out_stride, size)) && aligned(a->weight, 16) &&
                     aligned(a->codes, 8);
    return by_type<true>(a->type, A, vec, (hipStream_t)stream);
}
