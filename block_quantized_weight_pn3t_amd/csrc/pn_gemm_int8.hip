// pn_gemm_int8.hip -- products of 8-bit integers with a scale for each row of either side, on gfx950.
//
// out[m][n] = (sum_k a[m][k] w[n][k]) a_scales[m] w_scales[n]: exact sums in 32 bits on the matrix cores
// (16x16x64 instructions, rows of w as the rows of the result, so a lane ends with four neighbouring n of one
// m), scaled in fp32 as they are written. Integer sums have no order, so K may be cut in any way.
//
// Operands come from memory to LDS directly, 128 of K (a cache line of each row) at a time. A row's line lies in
// LDS as eight pieces of 16 bytes, piece p of row r at place p ^ (r & 7): a load writes a wave's 1 KB in a row,
// so the exchange is made in the addresses that it reads, and an instruction's operands of 16 rows come from
// all banks. Past the end of K the pieces are read from 16 zero bytes instead.
//
// Three kernels, by the number of tokens and of tiles:
//   stream  up to 32 tokens: memory bound, every weight read once. A workgroup has an even share of w's
//           rows; its waves share each tile of 32 rows by K and run on their own, several loads deep, until
//           their sums meet in LDS.
//   tile    tiles of 64 x 64 or 128 x 128, where there are too few of the next for all CUs; K is cut into parts
//           where there are too few of these, too, and a tile's last workgroup adds up (pn_arrive.h). (Even
//           shares of all tiles' lines for each workgroup were no faster: parts pass the caches by and are slow.)
//   large   tiles of 256 x 256: bound by the chip's power.
#include <math.h>

#include <algorithm>

#include "pn_arrive.h"
#include "pn_cache.h"
#include "pn_launch.h"

namespace pn {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

struct GemmArgs {
    const int8_t *a, *w;
    const float *a_scales, *w_scales;
    int64_t M, N, out_stride;
    int K;
    void *out;
    int tiles_m, tiles_n;  // of the outputs
    int splits;            // parts of K, of `each` lines
    int each;
    unsigned long long number;     // of the call (pn_arrive.h)
    unsigned long long *arrivals;  // [tile][kLine]
    unsigned long long *parts;     // [tile][part][numbers of a thread / 2][thread]
};

// 16 bytes that stand for K past its end.
__device__ const i32x4_t kZeros[1] = {{0, 0, 0, 0}};

// 16 bytes a lane from memory to LDS, a wave's in a row from lds on (ONCE: of lines that are read once). In assembly,
// since the compiler would have every read of LDS wait for every such load. (m0 is a reserved register: the compiler keeps
// nothing in it from one statement to another.)
template <bool ONCE = false>
__device__ __forceinline__ void load_lds(const int8_t *p, uint32_t lds)
{
    if constexpr (ONCE)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt" ::"s"(lds), "v"(p) : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory");
}

// An offset that is worked out where it is used, and not kept in a register for the whole loop.
__device__ __forceinline__ uint32_t here(uint32_t offset)
{
    asm volatile("" : "+v"(offset));
    return offset;
}

__device__ __forceinline__ void order() { __builtin_amdgcn_sched_barrier(0); }
__device__ __forceinline__ void barrier()
{
    order();
    __builtin_amdgcn_s_barrier();
    order();
}
// Waits until at most VM loads from memory are under way and (LGKM) all of LDS's.
template <int VM, bool LGKM>
__device__ __forceinline__ void wait()
{
    static_assert(VM < 64);
    order();
    __builtin_amdgcn_s_waitcnt((VM & 15) | 7 << 4 | (LGKM ? 0 : 15) << 8 | (VM >> 4) << 14);
    order();
}

__device__ __forceinline__ i32x4_t products(i32x4_t w, i32x4_t a, i32x4_t c)
{
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a, c, 0, 0, 0);
}

// ---- up to 32 tokens ------------------------------------------------------------------------------

// EIGHTS: eights of tokens that are loaded, 1, 2 or 4. 34816 x 5120 at one token 29 us (6.1 TB/s of weights; a copy
// reaches 4.9), at 16 31.7, 17 33.8, 32 38.3; 248320 x 5120 at four 214 (6.0); 5120 x 17408 at 13 16 (5.6), 32 21.8.
template <int EIGHTS>
struct Stream {
    static constexpr int WAVES = 4, ROWS = 32, TILES = (EIGHTS + 1) / 2;  // 16 tokens a tile
    static constexpr int STAGE = (ROWS + 8 * EIGHTS) * 128, LOADS = STAGE / 1024;
    static constexpr int STAGES = EIGHTS == 4 ? 3 : EIGHTS == 2 ? 5 : 4;
    static constexpr int ROW = ROWS + 4;                         // a token's sums in LDS, padded
    static constexpr int SUMS = WAVES * TILES * 16 * ROW * 4;    // bytes; twice, for every other tile
    static constexpr int MOST = 1024;                            // rows a workgroup has
    static constexpr int BYTES = WAVES * STAGES * STAGE + 2 * SUMS + (MOST + 32) * 4;
};

template <int T, int EIGHTS, bool ONCE>
__global__ void __launch_bounds__(256) gemm_int8_stream_kernel(GemmArgs A)
{
    typedef Stream<EIGHTS> S;
    typedef typename Elem<T>::type E;
    extern __shared__ i32x4_t lds[];
    char *const base = reinterpret_cast<char *>(lds);
    int *const sums = reinterpret_cast<int *>(base + S::WAVES * S::STAGES * S::STAGE);
    float *const scales = reinterpret_cast<float *>(base + S::WAVES * S::STAGES * S::STAGE + 2 * S::SUMS);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    // an even share of the rows
    const int64_t share = A.N / gridDim.x, more = A.N % gridDim.x;
    const int64_t n0 = blockIdx.x * share + min((int64_t)blockIdx.x, more);
    const int rows = (int)share + (blockIdx.x < more);
    const int tiles = (rows + S::ROWS - 1) / S::ROWS, steps = ((A.K + 127) / 128 + S::WAVES - 1) / S::WAVES;
    for (int i = threadIdx.x; i < rows; i += 256)
        scales[i] = A.w_scales[n0 + i];
    if (threadIdx.x < 32)
        scales[S::MOST + threadIdx.x] = A.a_scales[min((int64_t)threadIdx.x, A.M - 1)];

    const int r = lane >> 3, piece = (lane & 7) ^ r;
    const uint32_t stages = (uint32_t)(uintptr_t)lds + wave * S::STAGES * S::STAGE;
    // the next load: its tile's first row, its line of K and its stage
    int next_row = 0, next_step = 0, next_stage = 0;
    const auto load = [&]() {
        const int k = (next_step * S::WAVES + wave) * 128 + 16 * piece;
        const bool in = k < A.K && next_row < rows;
        const uint32_t to = stages + next_stage * S::STAGE;
#pragma unroll
        for (int j = 0; j < S::ROWS / 8; j++)
            load_lds<ONCE>(in ? A.w + (n0 + min(next_row + 8 * j + r, rows - 1)) * A.K + k : reinterpret_cast<const int8_t *>(kZeros),
                           to + j * 1024);
#pragma unroll
        for (int j = 0; j < EIGHTS; j++)
            load_lds(in ? A.a + min(8 * j + r, (int)A.M - 1) * A.K + k : reinterpret_cast<const int8_t *>(kZeros),
                     to + (S::ROWS / 8 + j) * 1024);
        if (++next_step == steps) {
            next_step = 0;
            next_row += S::ROWS;
        }
        if (++next_stage == S::STAGES)
            next_stage = 0;
    };

    __syncthreads();
#pragma unroll
    for (int i = 0; i < S::STAGES - 1; i++)
        load();
    const int row = lane & 15, g = lane >> 4;
    const uint32_t first_w = row * 128 + (g ^ (lane & 7)) * 16;
    const uint32_t first_a = S::ROWS * 128 + (EIGHTS == 1 ? row & 7 : row) * 128 + (g ^ (lane & 7)) * 16;
    int stage = 0;
    for (int tile = 0; tile < tiles; tile++) {
        i32x4_t acc[2][S::TILES] = {};
        for (int step = 0; step < steps; step++) {
            wait<63, true>();  // what is overwritten has been read
            load();
            wait<(S::STAGES - 1) * S::LOADS, false>();
            const char *const p = base + (wave * S::STAGES + stage) * S::STAGE;
#pragma unroll
            for (int t = 0; t < 2; t++) {
                i32x4_t fw[2], fa[S::TILES];
#pragma unroll
                for (int i = 0; i < 2; i++)
                    fw[i] = *reinterpret_cast<const i32x4_t *>(p + (first_w ^ 64 * t) + i * 2048);
#pragma unroll
                for (int i = 0; i < S::TILES; i++)
                    fa[i] = *reinterpret_cast<const i32x4_t *>(p + (first_a ^ 64 * t) + i * 2048);
#pragma unroll
                for (int i = 0; i < 2; i++)
#pragma unroll
                    for (int j = 0; j < S::TILES; j++)
                        acc[i][j] = products(fw[i], fa[j], acc[i][j]);
            }
            if (++stage == S::STAGES)
                stage = 0;
        }
        // the waves' sums: [wave][token][row]; the tile after next has the same place, behind another barrier
        int *const mine = sums + (tile & 1) * (S::SUMS / 4);
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int j = 0; j < S::TILES; j++)
                *reinterpret_cast<i32x4_t *>(mine + ((wave * S::TILES + j) * 16 + row) * S::ROW + 16 * i + 4 * g) = acc[i][j];
        wait<63, true>();
        barrier();
#pragma unroll
        for (int i = 0; i < S::TILES * 2; i++) {
            const int m = i * 8 + (int)(threadIdx.x >> 5), n = (int)threadIdx.x & 31, at = tile * S::ROWS + n;
            int sum = 0;
#pragma unroll
            for (int v = 0; v < S::WAVES; v++)
                sum += mine[(v * S::TILES * 16 + m) * S::ROW + n];
            if (m < A.M && at < rows)
                reinterpret_cast<E *>(A.out)[m * A.out_stride + n0 + at] = (E)((float)sum * scales[S::MOST + m] * scales[at]);
        }
    }
    wait<0, true>();
}

// ---- tiles ----------------------------------------------------------------------------------------

// Which tile a workgroup has. Workgroups go to the eight XCDs in turn, each with its own second-level cache:
// each XCD gets a run of tiles, in bands of kBand rows of tiles, down a band's column first, so that the tiles that
// an XCD works on share their rows of either operand.
constexpr int kBand = 4;
__device__ __forceinline__ void tile_of(const GemmArgs &A, int block, int blocks, int &tm, int &tn)
{
    const int xcd = block & 7, each = blocks >> 3, more = blocks & 7;
    const int at = xcd * each + min(xcd, more) + (block >> 3);
    const int band = at / (kBand * A.tiles_n), in = at - band * kBand * A.tiles_n;
    const int high = min(kBand, A.tiles_m - band * kBand);
    const int column = in / high;  // a division runs on the vector unit
    tn = __builtin_amdgcn_readfirstlane(column);
    tm = __builtin_amdgcn_readfirstlane(band * kBand + in - column * high);
}

// SIZE x SIZE outputs a workgroup, a quarter each wave. A line of K takes 0.25 us (64, one workgroup a CU) and 0.5 (128). Bound by
// its loads, from the Infinity Cache or memory, three or seven lines ahead: 777 x 1024 x 5120 13.4 us, 12.1 without the products
// and LDS reads of the loop, 9.8 without its loads; 300 x 5120 x 5120 20.0, 19.5, 11.3; 256 x 5120 x 17408 (128) 41.9, 42.1, 25.3.
template <int SIZE, int STAGES_>
struct Square {
    static constexpr int STAGE = 2 * SIZE * 128, LOADS = STAGE / 4096, STAGES = STAGES_;
    static constexpr int BYTES = STAGES * STAGE, N = SIZE / 32;  // 16-row tiles of a wave, each way
    static_assert(LOADS == 2 * N);
};

template <int T, int SIZE, int STAGES>
__global__ void __launch_bounds__(256) gemm_int8_tile_kernel(GemmArgs A)
{
    typedef Square<SIZE, STAGES> S;
    typedef typename Elem<T>::type E;
    typedef E E4 __attribute__((ext_vector_type(4)));
    typedef E E4Any __attribute__((ext_vector_type(4), aligned(sizeof(E))));  // rows of out of any alignment
    extern __shared__ i32x4_t lds[];  // [stage][a, w][row][piece]
    __shared__ bool last;
    char *const base = reinterpret_cast<char *>(lds);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int tiles = A.tiles_m * A.tiles_n, part = (int)blockIdx.x / tiles;
    int tm, tn;
    tile_of(A, (int)blockIdx.x - part * tiles, tiles, tm, tn);
    const int64_t m0 = (int64_t)tm * SIZE, n0 = (int64_t)tn * SIZE;

    const int r = threadIdx.x >> 3, piece = (lane & 7) ^ (r & 7);
    const int8_t *const a0 = A.a + m0 * A.K, *const w0 = A.w + n0 * A.K;
    const int last_a = (int)min(A.M - 1 - m0, (int64_t)SIZE - 1), last_w = (int)min(A.N - 1 - n0, (int64_t)SIZE - 1);
    uint32_t src[2][S::N];
#pragma unroll
    for (int j = 0; j < S::N; j++) {
        src[0][j] = (uint32_t)(min(r + 32 * j, last_a) * A.K + 16 * piece);
        src[1][j] = (uint32_t)(min(r + 32 * j, last_w) * A.K + 16 * piece);
    }
    const uint32_t stages = (uint32_t)(uintptr_t)lds + wave * 1024;
    const int first = part * A.each, end = min((A.K + 127) / 128, first + A.each);
    // load n of a step: the first half of them are a's rows
    const auto load = [&](int step, int stage, int n) {
        const int k = step < end ? step * 128 : A.K, o = n / S::N, j = n % S::N;
        const bool in = k + 16 * piece < A.K;
        load_lds(in ? (o ? w0 : a0) + k + src[o][j] : reinterpret_cast<const int8_t *>(kZeros),
                 stages + stage * S::STAGE + o * SIZE * 128 + j * 4096);
    };
#pragma unroll
    for (int i = 0; i < S::STAGES; i++)
#pragma unroll
        for (int n = 0; n < S::LOADS; n++)
            load(first + i, i, n);
    const int row = lane & 15, g = lane >> 4, wm = (wave & 1) * (SIZE / 2), wn = (wave >> 1) * (SIZE / 2);
    const uint32_t first_a = (wm + row) * 128 + (g ^ (lane & 7)) * 16, first_w = (SIZE + wn + row) * 128 + (g ^ (lane & 7)) * 16;
    i32x4_t fa[2][S::N][2], fw[2][S::N][2];  // [step & 1]: one is read while the other is multiplied
    const auto read = [&](int stage, int to, int i, int t) {
        const char *const p = base + stage * S::STAGE;
        fa[to][i][t] = *reinterpret_cast<const i32x4_t *>(p + (first_a ^ 64 * t) + i * 2048);
        fw[to][i][t] = *reinterpret_cast<const i32x4_t *>(p + (first_w ^ 64 * t) + i * 2048);
    };
    i32x4_t acc[S::N][S::N] = {};  // [16 of m][16 of n]
    wait<(S::STAGES - 1) * S::LOADS, true>();
    barrier();
#pragma unroll
    for (int t = 0; t < 2; t++)
#pragma unroll
        for (int i = 0; i < S::N; i++)
            read(0, 0, i, t);
    int stage = 0;
    const auto one = [&](int step, int from) {
        wait<(S::STAGES - 2) * S::LOADS, true>();  // the next step has landed, this one has been read
        barrier();
        const int to = stage;
        stage = stage + 1 == S::STAGES ? 0 : stage + 1;
        // one wave a SIMD: products, reads of the next step and loads in turn keep all three under way
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int i = 0; i < S::N; i++) {
                read(stage, from ^ 1, i, t);
                load(step + S::STAGES, to, t * S::N + i);
#pragma unroll
                for (int j = 0; j < S::N; j++)
                    acc[i][j] = products(fw[from][j][t], fa[from][i][t], acc[i][j]);
                order();
            }
        // (used here, or the compiler moves the reads to where the next step begins)
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int i = 0; i < S::N; i++)
                asm volatile("" : "+v"(fa[from ^ 1][i][t]), "+v"(fw[from ^ 1][i][t]));
    };
    for (int step = first; step < end; step += 2) {
        one(step, 0);
        if (step + 1 < end)
            one(step + 1, 1);
    }
    wait<0, true>();
    if (A.splits > 1) {
        const int tile = tm * A.tiles_n + tn;
        constexpr int NUMBERS = S::N * S::N * 2;  // of 64 bits
        unsigned long long *const parts = A.parts + (int64_t)tile * A.splits * NUMBERS * 256 + threadIdx.x;
#pragma unroll
        for (int i = 0; i < S::N; i++)
#pragma unroll
            for (int j = 0; j < S::N; j++)
#pragma unroll
                for (int e = 0; e < 2; e++)
                    put_shared(parts + ((int64_t)part * NUMBERS + (i * S::N + j) * 2 + e) * 256,
                               (unsigned long long)(uint32_t)acc[i][j][2 * e + 1] << 32 | (uint32_t)acc[i][j][2 * e]);
        wait<0, false>();  // every wave's, before the barrier
        __syncthreads();
        if (threadIdx.x == 0)
            last = arrive_last(A.arrivals + (int64_t)tile * kLine, A.number, (unsigned)A.splits);
        __syncthreads();
        if (!last)
            return;
        for (int other = 0; other < A.splits; other++) {
            if (other == part)
                continue;
#pragma unroll
            for (int i = 0; i < S::N; i++)
#pragma unroll
                for (int j = 0; j < S::N; j++)
#pragma unroll
                    for (int e = 0; e < 2; e++) {
                        const unsigned long long v = get_shared(parts + ((int64_t)other * NUMBERS + (i * S::N + j) * 2 + e) * 256);
                        acc[i][j][2 * e] += (int)(uint32_t)v;
                        acc[i][j][2 * e + 1] += (int)(v >> 32);
                    }
        }
    }
    float sw[S::N][4];
#pragma unroll
    for (int j = 0; j < S::N; j++)
#pragma unroll
        for (int e = 0; e < 4; e++)
            sw[j][e] = A.w_scales[min(n0 + wn + 16 * j + 4 * g + e, A.N - 1)];
#pragma unroll
    for (int i = 0; i < S::N; i++) {
        const int64_t m = m0 + wm + 16 * i + row;
        if (m >= A.M)
            continue;
        const float sa = A.a_scales[m];
#pragma unroll
        for (int j = 0; j < S::N; j++) {
            const int64_t n = n0 + wn + 16 * j + 4 * g;
            E *const p = reinterpret_cast<E *>(A.out) + m * A.out_stride + n;
            E4 v;
#pragma unroll
            for (int e = 0; e < 4; e++)
                v[e] = (E)((float)acc[i][j][e] * sa * sw[j][e]);
            if (n + 4 <= A.N) {
                *reinterpret_cast<E4Any *>(p) = v;
            } else {
#pragma unroll
                for (int e = 0; e < 4; e++)
                    if (n + e < A.N)
                        p[e] = v[e];
            }
        }
    }
}

// ---- 256 x 256 ------------------------------------------------------------------------------------

constexpr int kUnit = 128 * 128;  // bytes of a half of either operand's rows, a line each
constexpr int kLargeBytes = 8 * kUnit;

// Eight waves of 128 x 64 outputs each, two waves a SIMD, which alternate: while one multiplies, the other reads its
// operands and starts loads, a barrier between. A line of K is four such turns, one for each pair of halves of
// the wave's rows: (A0, B0), (A0, B1), (A1, B1), (A1, B0). What a turn reads can be loaded over two turns
// later, when both waves have read it, and so each unit is loaded a step and a half before it is read.
//
// 8192 x 34816 x 5120, bf16: 1.07 to 1.11 ms over several boxes, 2.6 to 2.7 POP/s; the matrix unit is busy 70 % of the time at the 1.75 GHz to which the
// chip lowers its clock (2.4 GHz with 16 tiles, where a line takes 0.96 us, 0.85 at the unit's rate). Without the
// alternation, reads among the products and one barrier a turn, 1.21 ms; with 32x32x32 instructions, of which a turn has
// two chains only, 1.34; without loads 0.90, without LDS reads 0.97.
template <int T>
__global__ void __launch_bounds__(512, 2) gemm_int8_large_kernel(GemmArgs A)
{
    extern __shared__ i32x4_t lds[];  // [step & 1][A0, A1, B0, B1][128 rows][8 pieces]
    typedef typename Elem<T>::type E;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wr = wave & 1, wc = wave >> 1;  // waves w and w + 4 share a SIMD
    int tm, tn;
    tile_of(A, (int)blockIdx.x, A.tiles_m * A.tiles_n, tm, tn);
    const int64_t m0 = (int64_t)tm * 256, n0 = (int64_t)tn * 256;

    // loading: a thread has a piece of rows t / 8 and t / 8 + 64 of each unit
    const int piece = (threadIdx.x & 7) ^ ((threadIdx.x >> 3) & 7);
    const int8_t *const a0 = A.a + m0 * A.K, *const w0 = A.w + n0 * A.K;
    const int last_a = (int)min(A.M - 1 - m0, (int64_t)255), last_w = (int)min(A.N - 1 - n0, (int64_t)255);
    uint32_t src[4][2];
#pragma unroll
    for (int j = 0; j < 2; j++) {
        const int r = (int)(threadIdx.x >> 3) + 64 * j;
#pragma unroll
        for (int h = 0; h < 2; h++) {
            src[h][j] = (uint32_t)(min((r >> 6) * 128 + h * 64 + (r & 63), last_a) * A.K + 16 * piece);
            src[2 + h][j] = (uint32_t)(min((r >> 5) * 64 + h * 32 + (r & 31), last_w) * A.K + 16 * piece);
        }
    }
    const uint32_t lds_base = (uint32_t)(uintptr_t)lds + wave * 1024;
    const auto load = [&](int step, int unit) {
        const int k = step * 128;
        const bool in = k + 16 * piece < A.K;
        const int8_t *const base = (unit < 2 ? a0 : w0) + k;
#pragma unroll
        for (int j = 0; j < 2; j++)
            load_lds(in ? base + src[unit][j] : reinterpret_cast<const int8_t *>(kZeros),
                     lds_base + ((step & 1) * 4 + unit) * kUnit + j * 8192);
    };

    i32x4_t fa[4][2], fb[2][2][2];
    const int row = lane & 15, g = lane >> 4;
    // a lane's first piece of its row; the other is four pieces on, before the exchange of pieces
    const uint32_t first_a = (wr * 64 + row) * 128 + (g ^ (lane & 7)) * 16, first_b = (wc * 32 + row) * 128 + (g ^ (lane & 7)) * 16;
    const auto piece_at = [&](uint32_t first, int buffer, int t, int at) {
        return *reinterpret_cast<const i32x4_t *>(reinterpret_cast<const char *>(lds) + ((first ^ 64 * t) + buffer * 4 * kUnit) + at);
    };
    const auto read_a = [&](int buffer, int h) {
        const uint32_t first = here(first_a);
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int i = 0; i < 4; i++)
                fa[i][t] = piece_at(first, buffer, t, h * kUnit + i * 2048);
    };
    const auto read_b = [&](int buffer, int h, int to) {
        const uint32_t first = here(first_b);
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int j = 0; j < 2; j++)
                fb[to][j][t] = piece_at(first, buffer, t, (2 + h) * kUnit + j * 2048);
    };
    i32x4_t acc[2][4][2][2] = {};  // [half of A][i][half of B][j]
    const auto multiply = [&](int ha, int hb, int from) {
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int t = 0; t < 2; t++)
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int j = 0; j < 2; j++)
                    acc[ha][i][hb][j] = products(fb[from][j][t], fa[i][t], acc[ha][i][hb][j]);
        __builtin_amdgcn_s_setprio(0);
        barrier();
    };
    // the end of a turn's reads: they are in registers, and what the next turn reads has landed (of the eight units
    // under way, the six last may be on their way)
    const auto landed = [&]() {
        wait<12, true>();
        barrier();
    };

    // units in the order in which they are read
#pragma unroll
    for (int step = 0; step < 2; step++) {
        load(step, 2);
        load(step, 0);
        load(step, 3);
        load(step, 1);
    }
    wait<12, false>();
    barrier();
    read_b(0, 0, 0);
    wait<63, true>();
    barrier();
    if (wave >= 4)  // the second wave of each SIMD is half a turn behind
        barrier();
    const int steps = (A.K + 127) / 128;
    const auto one = [&](int step, int buffer) {
        read_a(buffer, 0);
        load(step + 2, 2);
        landed();
        multiply(0, 0, buffer);
        read_b(buffer, 1, buffer ^ 1);
        load(step + 2, 0);
        landed();
        multiply(0, 1, buffer ^ 1);
        read_a(buffer, 1);
        load(step + 2, 3);
        landed();
        multiply(1, 1, buffer ^ 1);
        read_b(buffer ^ 1, 0, buffer ^ 1);  // the next step's
        load(step + 2, 1);
        landed();
        multiply(1, 0, buffer);
    };
    for (int step = 0; step < steps; step += 2) {
        one(step, 0);
        if (step + 1 < steps)
            one(step + 1, 1);
    }
    if (wave < 4)
        barrier();
    wait<0, true>();
    barrier();

    // A lane has token row of 16 and four rows of w, 4g .. 4g + 3: sixteen tokens at a time go through the wave's own
    // part of LDS to be written as whole lines. (Vectors at any address: 2846 x 14445 x 1024, bf16, 64 us, 116
    // by single numbers; 14448 wide 63.)
    constexpr int VEC = 16 / sizeof(E), LANES = 64 / VEC, STRIDE = 64 + VEC;  // lanes and elements a token's row of 64
    typedef E EV __attribute__((ext_vector_type(VEC)));
    typedef E EVAny __attribute__((ext_vector_type(VEC), aligned(sizeof(E))));  // rows of out of any alignment
    typedef E E4 __attribute__((ext_vector_type(4)));
    E *const stage = reinterpret_cast<E *>(lds) + wave * 16 * STRIDE;
    const int64_t n_wave = n0 + wc * 64, m_wave = m0 + wr * 128;
    float sw[2][2][4];
#pragma unroll
    for (int hb = 0; hb < 2; hb++)
#pragma unroll
        for (int j = 0; j < 2; j++)
#pragma unroll
            for (int e = 0; e < 4; e++)
                sw[hb][j][e] = A.w_scales[min(n_wave + hb * 32 + j * 16 + 4 * g + e, A.N - 1)];
#pragma unroll
    for (int ha = 0; ha < 2; ha++)
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const int64_t m = m_wave + ha * 64 + i * 16;
            if (m >= A.M)
                continue;
            const float sa = A.a_scales[min(m + row, A.M - 1)];
#pragma unroll
            for (int hb = 0; hb < 2; hb++)
#pragma unroll
                for (int j = 0; j < 2; j++) {
                    E4 v;
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        v[e] = (E)((float)acc[ha][i][hb][j][e] * sa * sw[hb][j][e]);
                    *reinterpret_cast<E4 *>(stage + row * STRIDE + hb * 32 + j * 16 + 4 * g) = v;
                }
#pragma unroll
            for (int q = 0; q < 16 * LANES / 64; q++) {
                const int at = q * (64 / LANES) + lane / LANES, c = lane % LANES * VEC;
                const EV v = *reinterpret_cast<const EV *>(stage + at * STRIDE + c);
                E *const p = reinterpret_cast<E *>(A.out) + (m + at) * A.out_stride + n_wave + c;
                if (m + at >= A.M)
                    continue;
                if (n_wave + c + VEC <= A.N) {
                    *reinterpret_cast<EVAny *>(p) = v;
                } else {
#pragma unroll
                    for (int e = 0; e < VEC; e++)
                        if (n_wave + c + e < A.N)
                            p[e] = v[e];
                }
            }
        }
}

// ---- host -----------------------------------------------------------------------------------------

static bool gemm_fit(int64_t M, int64_t N, int64_t K)
{
    return M >= 0 && N >= 0 && M <= INT32_MAX && N <= INT32_MAX && K >= 16 && K % 16 == 0 && K <= PN_GEMM_INT8_MAX_K &&
           ((M + 63) / 64) * ((N + 63) / 64) <= INT32_MAX / 64 &&
           ((M + 255) / 256) * ((N + 255) / 256) <= launch_most(512);  // so that tiles of 256 can always be launched
}

// How a product is cut.
struct GemmCut {
    int size;    // of a tile: 0 for the stream
    int splits;  // parts of K
    int each;    // lines of 128 of a part
    int64_t workspace;
};
static GemmCut gemm_cut(int64_t M, int64_t N, int64_t K)
{
    const auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
    const int64_t cus = device_cus(), lines = up(K, 128);
    GemmCut c = {};
    c.splits = 1;
    c.each = (int)lines;
    if (M <= 32)
        return c;
    // What is estimated to be soonest, in us: rounds of workgroups, each some time a line and some to begin and end,
    // and the joining of K's parts. Measured for a line: 0.25 and 0.38 with one and two workgroups a CU (64), 0.5
    // (128; half of it where a last round leaves most CUs idle), 0.92 (256). So 64 x 1024 x 5120 is four parts in tiles
    // of 64 (9.3 us; whole 11.7, in tiles of 128 19.9), 256 x 5120 x 17408 three in tiles of 128 (42; 82 whole, 61 in tiles
    // of 64), 1024 x 5120 x 5120 tiles of 128 (44; 49 in those of 256), 2048 x 6144 x 5120 tiles of 256 (57; 75 in those
    // of 128), 4096 x 5120 x 1024 too (35; 45), 777 x 5120 x 1024 tiles of 64 (15.9; 18.5 in those of 128).
    // The estimate has no term for the memory's rate, and a wide matrix that comes from memory gains nothing from idle CUs:
    // 96 and 128 x 34816 x 5120 go to tiles of 128 (67.1 and 71.5 us) where those of 256 take 58.5 and 61.3, x 4096 56.8 and
    // 59.9 for 47.4 and 49.4. Two parts in tiles of 128 would be sooner, too, than the tiles of 64 that 300 x 4096 x 6144,
    // 8896 and 12288 go to (22.3, 29.4, 34.2; 20.2, 25.2, 29.1), tiles of 128 than those of 256 for 1500 x 5120 x 6144
    // (56.6, 58.1).
    double best = INFINITY;
    for (const int size : {64, 128, 256}) {
        const int64_t t = up(M, size) * up(N, size), slots = size == 64 ? 2 * cus : cus;
        const double edge = size == 64 ? 2.3 : size == 128 ? 5.2 : 10.0;
        for (int splits = 1; splits <= (size == 256 ? 1 : std::min<int64_t>(8, lines / 4 + 1)); splits++) {
            const int64_t each = up(lines, splits), blocks = t * splits;
            if (up(lines, each) != splits || (splits > 1 && blocks > 2 * slots) || blocks > launch_most(size == 256 ? 512 : 256))
                continue;
            const double line = size == 64 ? (blocks <= cus ? 0.25 : 0.38) : size == 128 ? 0.5 : 0.92;
            const double join = splits == 1 ? 0.0 : size == 64 ? 2.3 + 0.6 * splits : 1.45 * splits;
            const int64_t idle = size == 128 && blocks > slots ? up(blocks, slots) * slots - blocks : 0;
            const double time = (double)up(blocks, slots) * ((double)each * line + edge) + join -
                                (double)each * 0.25 * (double)idle / (double)slots;
            if (time < best) {
                best = time;
                c.size = size;
                c.splits = splits;
                c.each = (int)each;
                c.workspace = splits > 1 ? t * (kLine * 8 + (int64_t)splits * size * size * 4) : 0;
            }
        }
    }
    return c;
}

// Launches kernel KERN with its dynamic LDS.
template <auto KERN>
static int launch_gemm(const GemmArgs &A, unsigned blocks, int threads, int bytes, hipStream_t s)
{
    if (!lds_limit_once<KERN>(bytes))
        return PN_ERR_HIP;
    hipLaunchKernelGGL(KERN, dim3(blocks), dim3(threads), bytes, s, A);
    return launch_status();
}

template <int T, bool ONCE>
static int run_stream(const GemmArgs &A, unsigned blocks, hipStream_t s)
{
    return A.M <= 8    ? launch_gemm<gemm_int8_stream_kernel<T, 1, ONCE>>(A, blocks, 256, Stream<1>::BYTES, s)
           : A.M <= 16 ? launch_gemm<gemm_int8_stream_kernel<T, 2, ONCE>>(A, blocks, 256, Stream<2>::BYTES, s)
                       : launch_gemm<gemm_int8_stream_kernel<T, 4, ONCE>>(A, blocks, 256, Stream<4>::BYTES, s);
}

template <int T>
static int run_gemm(GemmArgs A, const GemmCut &c, hipStream_t s)
{
    if (c.size == 0) {
        // One workgroup a CU, as many rows each as it takes. Weights that the memory's cache (256 MB) cannot keep beside
        // others until their next use pass it by: 178 MB 32.8 us, 35.3 through it; 89 MB, partly kept, 16.4 and 19.2 past.
        const int64_t cus = device_cus();
        const unsigned blocks = (unsigned)std::max(std::min((A.N + 7) / 8, cus), (A.N + 1023) / 1024);
        return A.N * A.K >= (int64_t)128 << 20 ? run_stream<T, true>(A, blocks, s) : run_stream<T, false>(A, blocks, s);
    }
    A.tiles_m = (int)((A.M + c.size - 1) / c.size);
    A.tiles_n = (int)((A.N + c.size - 1) / c.size);
    A.splits = c.splits;
    A.each = c.each;
    const unsigned blocks = (unsigned)A.tiles_m * A.tiles_n * c.splits;
    return c.size == 256   ? launch_gemm<gemm_int8_large_kernel<T>>(A, blocks, 512, kLargeBytes, s)
           : c.size == 128 ? launch_gemm<gemm_int8_tile_kernel<T, 128, 4>>(A, blocks, 256, Square<128, 4>::BYTES, s)
           : blocks <= (unsigned)device_cus()
               ? launch_gemm<gemm_int8_tile_kernel<T, 64, 8>>(A, blocks, 256, Square<64, 8>::BYTES, s)
               : launch_gemm<gemm_int8_tile_kernel<T, 64, 4>>(A, blocks, 256, Square<64, 4>::BYTES, s);
}

}  // namespace pn

using namespace pn;

extern "C" int64_t pn_gemm_int8_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (!gemm_fit(M, N, K) || M == 0 || N == 0 || K <= 3 * 128)
        return 0;
    // The most that any number of rows up to M takes, which all come down to multiples of 64: more rows can need less, as
    // their tiles are enough without parts of K (none has parts from `whole` rows on).
    const int64_t cus = device_cus(), whole = std::max(2 * cus / ((N + 63) / 64) * 64, cus / ((N + 127) / 128) * 128);
    int64_t most = 0;
    for (int64_t m = std::min(M, whole); m > 32; m = (m - 1) / 64 * 64)
        most = std::max(most, gemm_cut(m, N, K).workspace);
    return most;
}

extern "C" int pn_gemm_int8_cut(int64_t M, int64_t N, int64_t K, int *parts)
{
    if (!gemm_fit(M, N, K) || M == 0 || N == 0)
        return PN_ERR_SHAPE;
    const GemmCut c = gemm_cut(M, N, K);
    if (parts)
        *parts = c.splits;
    return c.size;
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
    const GemmCut c = gemm_cut(M, N, K);
    if (c.workspace > 0) {
        if (!workspace)
            return PN_ERR_NULL;
        if (!aligned(workspace, 16))
            return PN_ERR_ALIGN;
        if (workspace_bytes < c.workspace)
            return PN_ERR_WORKSPACE;
    }
    const int st = check_device();
    if (st != PN_OK)
        return st;
    GemmArgs A = {};
    A.a = a;
    A.w = w;
    A.a_scales = a_scales;
    A.w_scales = w_scales;
    A.M = M;
    A.N = N;
    A.out_stride = out_stride;
    A.K = (int)K;
    A.out = out;
    if (c.workspace > 0) {
        A.number = call_number();
        A.arrivals = (unsigned long long *)workspace;
        A.parts = A.arrivals + ((M + c.size - 1) / c.size) * ((N + c.size - 1) / c.size) * kLine;
    }
    hipStream_t s = (hipStream_t)stream;
    return type == PN_F32    ? run_gemm<PN_F32>(A, c, s)
           : type == PN_BF16 ? run_gemm<PN_BF16>(A, c, s)
                             : run_gemm<PN_F16>(A, c, s);
}
