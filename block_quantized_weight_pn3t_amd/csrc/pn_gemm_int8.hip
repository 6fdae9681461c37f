// pn_gemm_int8.hip -- products of 8-bit integers with a scale for each row of either side, on gfx950.
//
// out[m][n] = (sum_k a[m][k] w[n][k]) a_scales[m] w_scales[n]: exact sums in 32 bits on the matrix cores
// (16x16x64: 64 products a lane pair and instruction), scaled in fp32 as they are written.
//
// A workgroup of four waves has a tile of 64 x 64 outputs, a wave 32 x 32 of it; 64 of K at a time come
// through LDS.
#include "pn_cache.h"

namespace pn {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

struct GemmArgs {
    const int8_t *a, *w;
    const float *a_scales, *w_scales;
    int64_t M, N, out_stride;
    int K;
    void *out;
};

template <int T>
__global__ void __launch_bounds__(256) gemm_int8_kernel(GemmArgs A)
{
    __shared__ i32x4_t lds[2][64][5];  // rows of 64 bytes and 16 of padding
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
    const int r = threadIdx.x >> 2, c = threadIdx.x & 3;
    const int8_t *const pa = A.a + min(m0 + r, A.M - 1) * A.K + 16 * c;
    const int8_t *const pw = A.w + min(n0 + r, A.N - 1) * A.K + 16 * c;
    const int i = lane & 15, g = lane >> 4, wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
    i32x4_t acc[2][2] = {};
    for (int k = 0; k < A.K; k += 64) {
        const bool in = k + 16 * c < A.K;
        const i32x4_t va = in ? *reinterpret_cast<const i32x4_t *>(pa + k) : i32x4_t{0, 0, 0, 0};
        const i32x4_t vw = in ? *reinterpret_cast<const i32x4_t *>(pw + k) : i32x4_t{0, 0, 0, 0};
        __syncthreads();
        lds[0][r][c] = va;
        lds[1][r][c] = vw;
        __syncthreads();
#pragma unroll
        for (int y = 0; y < 2; y++)
#pragma unroll
            for (int x = 0; x < 2; x++)
                acc[y][x] = __builtin_amdgcn_mfma_i32_16x16x64_i8(lds[0][wm + 16 * y + i][g], lds[1][wn + 16 * x + i][g],
                                                                  acc[y][x], 0, 0, 0);
    }
#pragma unroll
    for (int x = 0; x < 2; x++) {
        const int64_t n = n0 + wn + 16 * x + i;
        if (n >= A.N)
            continue;
        const float sw = A.w_scales[n];
#pragma unroll
        for (int y = 0; y < 2; y++)
#pragma unroll
            for (int e = 0; e < 4; e++) {
                const int64_t m = m0 + wm + 16 * y + 4 * g + e;
                if (m < A.M)
                    reinterpret_cast<typename Elem<T>::type *>(A.out)[m * A.out_stride + n] =
                        (typename Elem<T>::type)((float)acc[y][x][e] * A.a_scales[m] * sw);
            }
    }
}

static bool gemm_fit(int64_t M, int64_t N, int64_t K)
{
    return M >= 0 && N >= 0 && M <= 65535 * 64 && N <= INT32_MAX && K >= 16 && K % 16 == 0 && K <= PN_GEMM_INT8_MAX_K;
}

}  // namespace pn

using namespace pn;

extern "C" int64_t pn_gemm_int8_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    return 0;
}

extern "C" int pn_gemm_int8(const int8_t *a, const float *a_scales, int64_t M, const int8_t *w,
                            const float *w_scales, int64_t N, int64_t K, int type, void *out,
                            int64_t out_stride, void *workspace, int64_t workspace_bytes, void *stream)
{
    const int size = elem_bytes(type);
    if (size == 0)
        return PN_ERR_FORMAT;
    if (!gemm_fit(M, N, K))
        return PN_ERR_SHAPE;
    if (M == 0 || N == 0)
        return PN_OK;
    if (!a || !a_scales || !w || !w_scales || !out)
        return PN_ERR_NULL;
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a_scales, 4) || !aligned(w_scales, 4) || !aligned(out, size))
        return PN_ERR_ALIGN;
    const int st = check_device();
    if (st != PN_OK)
        return st;
    const GemmArgs A{a, w, a_scales, w_scales, M, N, out_stride, (int)K, out};
    const dim3 grid((unsigned)((N + 63) / 64), (unsigned)((M + 63) / 64));
    hipStream_t s = (hipStream_t)stream;
    if (type == PN_F32)
        hipLaunchKernelGGL((gemm_int8_kernel<PN_F32>), grid, dim3(256), 0, s, A);
    else if (type == PN_BF16)
        hipLaunchKernelGGL((gemm_int8_kernel<PN_BF16>), grid, dim3(256), 0, s, A);
    else
        hipLaunchKernelGGL((gemm_int8_kernel<PN_F16>), grid, dim3(256), 0, s, A);
    return launch_status();
}
