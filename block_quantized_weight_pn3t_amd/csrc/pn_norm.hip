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
// Codes are those of the definition in 64 bits, computed in 32: 127 / T and its product are off by less than 5e-5
// there, and only where a quotient lies that near to a border between two codes (one number in ten thousand) is it
// worked out in 64 bits. T has to be exact for that: a product of two 16-bit numbers is in fp32, one with an fp32
// number is taken in 64 bits. Squares are summed in 64 bits.
//
// Measured: 8192 rows of 5120 bf16 with their residual to 8-bit rows 62 us (4.8 TB/s; a copy reaches 4.9), all of it in 64
// bits 99; 4095 of 17408 bf16 to 8-bit rows 45 us (4.8); four of 5120 fp32 4.1 us.
#include <float.h>

#include <algorithm>

#include "pn_cache.h"
#include "pn_lanes.h"
#include "pn_launch.h"

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


constexpr int VEC = 8;  // elements a thread loads at a time

// The elements from p[at] on that a row of K has, zeros past its end. Rows may begin anywhere: the type says that a
// load of 16 bytes is aligned to an element only, which the memory takes.
template <int T, bool WHOLE>
__device__ __forceinline__ void load_n(const void *p, int64_t row, int at, int K, float (&x)[VEC])
{
    typedef typename Elem<T>::type E;
    typedef E EN __attribute__((ext_vector_type(VEC), aligned(sizeof(E))));
    const E *const q = reinterpret_cast<const E *>(p) + row + at;
    if (WHOLE || at + VEC <= K) {
        const EN v = *reinterpret_cast<const EN *>(q);
#pragma unroll
        for (int j = 0; j < VEC; j++)
            x[j] = (float)v[j];
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j++)
            x[j] = at + j < K ? (float)q[j] : 0.0f;
    }
}
template <int T, bool WHOLE>
__device__ __forceinline__ void store_n(void *p, int64_t row, int at, int K, const float (&x)[VEC])
{
    typedef typename Elem<T>::type E;
    typedef E EN __attribute__((ext_vector_type(VEC), aligned(sizeof(E))));
    E *const q = reinterpret_cast<E *>(p) + row + at;
    EN v;
#pragma unroll
    for (int j = 0; j < VEC; j++)
        v[j] = (E)x[j];
    if (WHOLE || at + VEC <= K) {
        *reinterpret_cast<EN *>(q) = v;
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j++)
            if (at + j < K)
                q[j] = v[j];
    }
}

// Weights, of any type.
template <bool WHOLE>
__device__ __forceinline__ void load_weight(const NormArgs &A, int at, float (&w)[VEC])
{
    if (A.weight_type == PN_F32)
        load_n<PN_F32, WHOLE>(A.weight, 0, at, A.K, w);
    else if (A.weight_type == PN_BF16)
        load_n<PN_BF16, WHOLE>(A.weight, 0, at, A.K, w);
    else
        load_n<PN_F16, WHOLE>(A.weight, 0, at, A.K, w);
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu; }
constexpr uint32_t kInf = 0x7F800000u;  // magnitudes from here on are not finite

// What a row's lanes have found: the sum of squares, the largest |t| and its bits in fp32, numbers that are not finite.
struct Found {
    double ss, top;
    uint32_t bits;
    int bad;
};

// The same for all lanes of the row; `lds` is free where `again`.
template <bool WAVE>
__device__ __forceinline__ Found over_row(Found f, Found (&lds)[16], bool again)
{
    f.ss = over_lanes_sum(f.ss);
    f.top = over_lanes_max(f.top);
    f.bits = over_lanes_max(f.bits);
    f.bad = __any(f.bad);
    if constexpr (!WAVE) {
        if (again)
            __syncthreads();
        if ((threadIdx.x & 63) == 0)
            lds[threadIdx.x >> 6] = f;
        __syncthreads();
        // sixteen lanes have sixteen waves
        const int v = threadIdx.x & 15;
        f = v < (int)blockDim.x >> 6 ? lds[v] : Found{0.0, 0.0, 0, 0};
        const auto join = [&](auto mask) {
            constexpr int M = mask.value;
            f.ss += __builtin_bit_cast(double, moved_by<M>(__builtin_bit_cast(u64, f.ss)));
            f.top = fmax(f.top, __builtin_bit_cast(double, moved_by<M>(__builtin_bit_cast(u64, f.top))));
            f.bits = max(f.bits, moved_by<M>(f.bits));
        };
        join(std::integral_constant<int, 1>());
        join(std::integral_constant<int, 2>());
        join(std::integral_constant<int, 4>());
        join(std::integral_constant<int, 8>());
        f.bad = __any(f.bad);
    }
    return f;
}

enum { ROWS_ONLY, NORM_SHORT, NORM_LONG };

// MODE: the numbers' 8-bit rows alone, or the norm with products that are exact in fp32 or (LONG) may not be. NV: pieces
// of VEC elements a thread holds. WAVE: a wave a row. WHOLE: K is a multiple of VEC.
template <int T, int MODE, int NV, bool WAVE, bool WHOLE>
__global__ void __launch_bounds__(1024) norm_kernel(NormArgs A)
{
    __shared__ Found lds[16];
    constexpr bool NORM = MODE != ROWS_ONLY;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int threads = WAVE ? 64 : (int)blockDim.x, thread = WAVE ? lane : (int)threadIdx.x;
    const int64_t row = WAVE ? (int64_t)blockIdx.x * (blockDim.x >> 6) + wave : (int64_t)blockIdx.x;
    if (WAVE && row >= A.rows)
        return;

    float h[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int at = (i * threads + thread) * VEC;
        if (at < A.K)
            load_n<T, WHOLE>(A.x, row * A.x_stride, at, A.K, h[i]);
    }
    if (NORM && A.residual) {
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int at = (i * threads + thread) * VEC;
            if (at < A.K) {
                float r[VEC];
                load_n<T, WHOLE>(A.residual, row * A.residual_stride, at, A.K, r);
#pragma unroll
                for (int j = 0; j < VEC; j++)
                    h[i][j] = (float)(typename Elem<T>::type)(h[i][j] + r[j]);
            }
        }
    }
    // the weights stay in registers where there is room, else they are read again (from the caches)
    constexpr bool HOLD = NV * VEC <= 32;
    float held[HOLD ? NV : 1][VEC];
    Found f{0.0, 0.0, 0, 0};
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int at = (i * threads + thread) * VEC;
        if (at >= A.K)
            continue;
        float (&w)[VEC] = held[HOLD ? i : 0];
        if constexpr (NORM) {
            if (A.sum)
                store_n<T, WHOLE>(A.sum, row * A.sum_stride, at, A.K, h[i]);
            load_weight<WHOLE>(A, at, w);
        }
#pragma unroll
        for (int j = 0; j < VEC; j++) {
            if constexpr (NORM) {
                const double d = (double)h[i][j];
                f.ss = fma(d, d, f.ss);
            }
            if constexpr (MODE == ROWS_ONLY)
                f.bits = max(f.bits, magnitude(h[i][j]));
            if constexpr (MODE == NORM_SHORT)
                f.bits = max(f.bits, magnitude(h[i][j] * w[j]));
            if constexpr (MODE == NORM_LONG) {
                f.top = fmax(f.top, fabs((double)h[i][j] * (double)w[j]));
                f.bad |= magnitude(h[i][j]) >= kInf || magnitude(w[j]) >= kInf;
            }
        }
    }
    f = over_row<WAVE>(f, lds, false);
    double top = f.top;
    int none = f.bad;
    if constexpr (MODE != NORM_LONG) {
        top = (double)__builtin_bit_cast(float, f.bits);
        none = f.bits >= kInf;
    }
    // fp32 products that passed its range, or fell below it
    if (MODE == NORM_SHORT && !(top > 0x1p-100 && top < 0x1p100)) {
        Found g{0.0, 0.0, 0, 0};
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int at = (i * threads + thread) * VEC;
            if (at >= A.K)
                continue;
            float w[VEC];
            load_weight<WHOLE>(A, at, w);
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                g.top = fmax(g.top, fabs((double)h[i][j] * (double)w[j]));
                g.bad |= magnitude(h[i][j]) >= kInf || magnitude(w[j]) >= kInf;
            }
        }
        g = over_row<WAVE>(g, lds, true);
        top = g.top;
        none = g.bad;
    }

    double r = 1.0;
    if (NORM && (A.out || thread == 0))
        r = 1.0 / sqrt(f.ss / A.K + (double)A.eps);
    if (A.scales && thread == 0)
        A.scales[row] = none || !(r < INFINITY) ? __builtin_nanf("") : (float)(top * r / 127.0);
    const bool zero = none || !(top > 0.0), plain = top > 0x1p-100 && top < 0x1p100;
    const float inv = plain ? 127.0f / (float)top : 0.0f;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int at = (i * threads + thread) * VEC;
        if (at >= A.K)
            continue;
        float (&w)[VEC] = held[HOLD ? i : 0];
        if constexpr (NORM) {
            if (!HOLD)
                load_weight<WHOLE>(A, at, w);
            if (A.out) {
                float y[VEC];
#pragma unroll
                for (int j = 0; j < VEC; j++)
                    y[j] = to_f32((double)h[i][j] * r * (double)w[j]);
                store_n<T, WHOLE>(A.out, row * A.out_stride, at, A.K, y);
            }
        }
        if (A.codes) {
            uint32_t c[VEC];  // a code in the low byte of each
            float worst = 0.0f;
#pragma unroll
            for (int j = 0; j < VEC; j++) {
                // the sum with 1.5 * 2^23 has the nearest whole number in its low bits
                const float q = (NORM ? h[i][j] * w[j] : h[i][j]) * inv, n = q + 0x1.8p23f;
                worst = fmaxf(worst, fabsf(q - (n - 0x1.8p23f)));
                c[j] = __builtin_bit_cast(uint32_t, n);
            }
            if (zero) {
#pragma unroll
                for (int j = 0; j < VEC; j++)
                    c[j] = 0;
            } else if (!plain || !(worst < 0.49995f)) {
#pragma unroll
                for (int j = 0; j < VEC; j++) {
                    const double t = NORM ? (double)h[i][j] * (double)w[j] : (double)h[i][j];
                    c[j] = (uint32_t)(int)rint((127.0 * t) / top);
                }
            }
            int8_t *const p = A.codes + row * A.K + at;
            if (WHOLE || at + VEC <= A.K) {
                const auto four = [&](int j) {
                    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[j + 3], c[j + 2], 0x0c0c0400u),
                                                 __builtin_amdgcn_perm(c[j + 1], c[j], 0x0c0c0400u), 0x05040100u);
                };
                typedef uint32_t u32x2a1 __attribute__((ext_vector_type(2), aligned(1)));
                *reinterpret_cast<u32x2a1 *>(p) = u32x2a1{four(0), four(4)};
            } else {
#pragma unroll
                for (int j = 0; j < VEC; j++)
                    if (at + j < A.K)
                        p[j] = (int8_t)c[j];
            }
        }
    }
}

// A's rows from `first` on.
template <int T>
static NormArgs rows_from(NormArgs A, int64_t first)
{
    typedef typename Elem<T>::type E;
    const auto from = [first](auto *p, int64_t stride) { return p ? p + first * stride : p; };
    A.rows -= first;
    A.x = from((const E *)A.x, A.x_stride);
    A.residual = from((const E *)A.residual, A.residual_stride);
    A.sum = from((E *)A.sum, A.sum_stride);
    A.out = from((E *)A.out, A.out_stride);
    A.codes = from(A.codes, A.K);
    A.scales = from(A.scales, 1);
    return A;
}

template <int T, int MODE, int NV, bool WAVE>
static void launch_norm(NormArgs A, int pieces, hipStream_t s)
{
    const int per = WAVE ? 4 : 1, threads = WAVE ? 256 : ((pieces + NV - 1) / NV + 63) / 64 * 64;
    const int64_t most = launch_most(threads) * per;
    for (;; A = rows_from<T>(A, most)) {
        const dim3 grid((unsigned)((std::min(A.rows, most) + per - 1) / per)), block(threads);
        if (A.K % VEC == 0)
            hipLaunchKernelGGL((norm_kernel<T, MODE, NV, WAVE, true>), grid, block, 0, s, A);
        else
            hipLaunchKernelGGL((norm_kernel<T, MODE, NV, WAVE, false>), grid, block, 0, s, A);
        if (A.rows <= most)
            return;
    }
}

// A thread holds one piece where rows are few, for latency, or of fp32 (8192 rows of 5120, norm: one 120 us, two 128), and
// else two up to 8192 elements (bf16: one 72 us, two 63, four 72), four up to 32768.
template <int T, int MODE>
static int run_norm(const NormArgs &A, hipStream_t s)
{
    const int pieces = (A.K + VEC - 1) / VEC;
    if (pieces <= 64)
        launch_norm<T, MODE, 1, true>(A, pieces, s);
    else if (pieces <= 128)
        launch_norm<T, MODE, 2, true>(A, pieces, s);
    else if (pieces <= (T == PN_F32 || A.rows < 256 ? 1024 : 512))
        launch_norm<T, MODE, 1, false>(A, pieces, s);
    else if (pieces <= 1024)
        launch_norm<T, MODE, 2, false>(A, pieces, s);
    else if (pieces <= 4096)
        launch_norm<T, MODE, 4, false>(A, pieces, s);
    else
        launch_norm<T, MODE, 8, false>(A, pieces, s);
    return launch_status();
}

// Products of two 16-bit numbers are exact in fp32.
static int run_norm_of(int type, const NormArgs &A, hipStream_t s)
{
    const bool is_short = A.weight_type != PN_F32;
    return type == PN_F32    ? run_norm<PN_F32, NORM_LONG>(A, s)
           : type == PN_BF16 ? is_short ? run_norm<PN_BF16, NORM_SHORT>(A, s) : run_norm<PN_BF16, NORM_LONG>(A, s)
           : is_short        ? run_norm<PN_F16, NORM_SHORT>(A, s)
                             : run_norm<PN_F16, NORM_LONG>(A, s);
}

// Rows and widths that the kernels take.
static bool rows_fit(int64_t rows, int64_t K)
{
    return rows >= 0 && rows <= INT32_MAX && K >= 1 && K <= PN_ROW_MAX_WIDTH;
}

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
    hipStream_t s = (hipStream_t)stream;
    return type == PN_F32    ? run_norm<PN_F32, ROWS_ONLY>(A, s)
           : type == PN_BF16 ? run_norm<PN_BF16, ROWS_ONLY>(A, s)
                             : run_norm<PN_F16, ROWS_ONLY>(A, s);
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
    return run_norm_of(a->type, A, (hipStream_t)stream);
}
