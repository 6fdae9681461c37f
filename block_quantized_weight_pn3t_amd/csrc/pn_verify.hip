// pn_verify.hip -- drafted tokens verified against the target's probabilities, on gfx950.
//
// Draft i stands iff all before it do and u_i q_i(x_i) < p_i(x_i); after a accepted drafts the next
// token is drawn from r = max(p_a - q_a, 0) (p_a after the last draft, or where r is zero) by
// inversion: the first t with r_0 + .. + r_t > u R. What is NaN or negative is no probability: its
// draft falls and its token has r = 0. Probabilities are fp32 at most, so u q is exact in 64 bits, and
// differences and sums are taken there: their rounding (2^-53 a step) is far below what separates two
// tokens.
//
// Memory bound: one row of p and one of q a sequence. The rows are too long for one workgroup (a
// single CU reads a small part of what the memory gives), so they are cut into chunks of kChunk, which
// up to 64 workgroups share: every wave works out the accepted count by itself (a lane a draft, one
// ballot), and each chunk's sums of r and of p go to the workspace. The workgroup that arrives last
// takes all its chunks' sums, finds the chunk in which the running sum passes u R and the token inside
// it. (As two kernels 13.0 us a call for one sequence, 10.8 so.)
//
// Arrivals are counted in a word of the workspace, which nobody clears beforehand: its upper 44 bits
// hold the call's number, anything else there counts as zero arrivals, and the last one to arrive
// leaves zero, so a replayed graph finds it as the first run did. (An arrival takes about 30 ns of its
// word's cache line, one after another: with 122 workgroups a sequence and the words of 32 sequences in
// two lines, 148 us instead of 14. So there are few, and a line a word.) Which workgroup is last changes
// nothing in the result. The sums are atomic stores and loads at the device's scope, as the eight
// XCDs' caches are not kept alike within a kernel: they pass those caches by, so all that is left to
// order is that a store is complete before the arrival is counted, by a wait, and that the loads come
// after the last arrival, by the barrier. (A release and an acquire at the device's scope promise the
// same in the language's terms, but the release writes the whole XCD's cache back: 32 sequences 19.5 us
// without, 48 with.)
#include <algorithm>
#include <atomic>

#include "pn_cache.h"

namespace pn {

constexpr int kChunk = 2048;        // numbers of a row a workgroup sums
constexpr int kPer = kChunk / 256;  // of those, a thread's
constexpr int kLine = 16;           // words of a cache line

struct VerifyArgs {
    const void *p, *q;
    int64_t p_stride, q_stride;
    const int32_t *draft, *n_draft;
    const float *u_accept, *u_sample;
    int64_t V;
    int K, chunks, groups;         // chunks of a row, workgroups of a sequence
    int32_t *tokens, *accepted;
    unsigned long long number;     // of the call, in the upper 44 bits
    unsigned long long *arrivals;  // [sequence][kLine]
    double2 *sums;                 // [sequence][chunk]: r, p
};

template <int T>
__device__ __forceinline__ double prob(const void *p, int64_t at)
{
    return (double)(float)reinterpret_cast<const typename Elem<T>::type *>(p)[at];
}

// r of one token: 0 where p or q is no probability, NaN or negative (p > q >= 0 leaves p positive)
__device__ __forceinline__ double rest(double p, double q) { return p > q && q >= 0.0 ? p - q : 0.0; }
__device__ __forceinline__ double positive(double p) { return p > 0.0 ? p : 0.0; }

// How a sequence's next token is drawn: rows of p and q (one < 0: no row of q), and the draft that a
// certain q takes out of p (-1: none).
struct Draw {
    int64_t p_row, q_row;
    int out;
};
__device__ __forceinline__ Draw draw_of(const VerifyArgs &A, int64_t b, int a, int n)
{
    Draw d;
    d.p_row = (b * (A.K + 1) + a) * A.p_stride;
    d.q_row = a < n && A.q ? (b * A.K + a) * A.q_stride : -1;
    d.out = a < n && !A.q ? A.draft[b * A.K + a] : -1;
    return d;
}
__device__ __forceinline__ int drafts_of(const VerifyArgs &A, int64_t b)
{
    return A.n_draft ? min(max(A.n_draft[b], 0), A.K) : A.K;
}

// v of another lane by a DPP move (0 where the move has no source).
template <int CTRL, int ROWS>
__device__ __forceinline__ double moved(double v)
{
    const uint2 w = __builtin_bit_cast(uint2, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w.x, CTRL, ROWS, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w.y, CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(double, make_uint2(lo, hi));
}
// The sum over this lane and those below it in the wave: within rows of 16 lanes, then the last lane of
// the row before into odd rows, then of the first half into the second.
__device__ __forceinline__ double wave_scan(double v)
{
    v += moved<0x111, 0xF>(v);  // row_shr 1
    v += moved<0x112, 0xF>(v);
    v += moved<0x114, 0xF>(v);
    v += moved<0x118, 0xF>(v);
    v += moved<0x142, 0xA>(v);  // row_bcast 15
    v += moved<0x143, 0xC>(v);  // row_bcast 31
    return v;
}
// Where a running sum over the workgroup's threads first passes a value: each thread tells the first of
// its own places that does (INT32_MAX: none) with the sum before it, and the last place that has
// anything (-1: none). `lds` is used once a kernel.
struct Found {
    int first, last;
    double before;
};
__device__ __forceinline__ Found find(int first, int last, double before, Found *lds)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const unsigned long long any = __ballot(first != INT32_MAX), has = __ballot(last >= 0);
    // the threads' places rise with the lanes
    if (any ? lane == __ffsll(any) - 1 : lane == 0) {
        lds[wave].first = first;
        lds[wave].before = before;
    }
    if (has ? lane == 63 - __clzll(has) : lane == 0)
        lds[wave].last = last;
    __syncthreads();
    Found f = lds[0];
#pragma unroll
    for (int w = 1; w < 4; w++) {
        if (f.first == INT32_MAX) {
            f.first = lds[w].first;
            f.before = lds[w].before;
        }
        f.last = max(f.last, lds[w].last);
    }
    return f;
}

__device__ __forceinline__ void put_sum(double2 *at, double2 v)
{
    __hip_atomic_store(&at->x, v.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(&at->y, v.y, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ double2 get_sum(const double2 *at)
{
    return make_double2(__hip_atomic_load(&at->x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT),
                        __hip_atomic_load(&at->y, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
}

// Counts one arrival of call `number` and returns how many there were with it.
__device__ __forceinline__ unsigned arrive(unsigned long long *word, unsigned long long number)
{
    constexpr unsigned long long count = (1ull << 20) - 1;
    unsigned long long old = __hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    // each turn another workgroup has arrived: at most as many turns as workgroups
    while ((old & ~count) != number)
        if (__hip_atomic_compare_exchange_strong(word, &old, number | 1, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                                 __HIP_MEMORY_SCOPE_AGENT))
            return 1;
    return (unsigned)((__hip_atomic_fetch_add(word, 1ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1) & count);
}

// The token after a accepted drafts of n, from all chunks' sums.
template <int T>
__device__ __forceinline__ void choose(const VerifyArgs &A, int64_t b, int n, int a)
{
    __shared__ double2 wsum[4];
    __shared__ double wmine[4];
    __shared__ Found lds[2][4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const double2 *const sums = A.sums + b * A.chunks;

    // each thread has a run of chunks
    const int each = (A.chunks + 255) / 256;
    const int c0 = min(A.chunks, (int)threadIdx.x * each), c1 = min(A.chunks, c0 + each);
    double r = 0.0, p = 0.0;
    for (int c = c0; c < c1; c++) {
        const double2 s = get_sum(sums + c);
        r += s.x;
        p += s.y;
    }
    const double scan_r = wave_scan(r), scan_p = wave_scan(p);
    if (lane == 63)
        wsum[wave] = make_double2(scan_r, scan_p);
    __syncthreads();
    const double all_r = (wsum[0].x + wsum[1].x) + (wsum[2].x + wsum[3].x);
    const bool whole = !(all_r > 0.0);  // r is zero everywhere: draw from p
    double total = 0.0, sum = whole ? scan_p - p : scan_r - r;
#pragma unroll
    for (int w = 0; w < 4; w++) {
        const double s = whole ? wsum[w].y : wsum[w].x;
        if (w < wave)
            sum += s;
        total += s;
    }
    int64_t token = -1;
    if (total > 0.0) {
        const double at = (double)A.u_sample[b] * total;
        // the first chunk that passes `at`; if none, the last that has anything
        double found = 0.0;
        int first = INT32_MAX, last = -1;
        for (int c = c0; c < c1; c++) {
            const double2 both = each == 1 ? make_double2(r, p) : get_sum(sums + c);
            const double s = whole ? both.y : both.x;
            if (s > 0.0) {
                last = c;
                if (first == INT32_MAX && sum + s > at) {
                    first = c;
                    found = sum;
                }
            }
            sum += s;
        }
        const Found chunk = find(first, last, found, lds[0]);
        const bool passed = chunk.first != INT32_MAX;
        const int64_t base = (int64_t)(passed ? chunk.first : chunk.last) * kChunk;

        // the chunk's numbers, kPer in a row a thread
        const Draw d = draw_of(A, b, a, n);
        double x[kPer], mine = 0.0;
#pragma unroll
        for (int k = 0; k < kPer; k++) {
            const int64_t t = base + threadIdx.x * kPer + k;
            x[k] = 0.0;
            if (t < A.V) {
                const double pt = prob<T>(A.p, d.p_row + t);
                const double qt = d.q_row < 0 ? 0.0 : prob<T>(A.q, d.q_row + t);
                x[k] = whole ? positive(pt) : t == d.out ? 0.0 : rest(pt, qt);
            }
        }
#pragma unroll
        for (int k = 0; k < kPer; k++)
            mine += x[k];
        const double scan = wave_scan(mine);
        if (lane == 63)
            wmine[wave] = scan;
        __syncthreads();
        sum = (passed ? chunk.before : 0.0) + (scan - mine);
#pragma unroll
        for (int w = 0; w < 3; w++)
            if (w < wave)
                sum += wmine[w];
        first = INT32_MAX;
        last = -1;
#pragma unroll
        for (int k = 0; k < kPer; k++) {
            const int t = threadIdx.x * kPer + k;
            sum += x[k];
            if (x[k] > 0.0) {
                last = t;
                if (passed && first == INT32_MAX && sum > at)
                    first = t;
            }
        }
        const Found place = find(first, last, 0.0, lds[1]);
        token = base + (place.first != INT32_MAX ? place.first : place.last);
    }
    if (threadIdx.x == 0)
        A.tokens[b * (A.K + 1) + a] = (int32_t)token;
}

template <int T>
__global__ void __launch_bounds__(256) verify_kernel(VerifyArgs A)
{
    typedef typename Elem<T>::type E;
    constexpr int VEC = 16 / sizeof(E);
    typedef E EV __attribute__((ext_vector_type(VEC)));
    __shared__ double2 lds[2][4];  // of even and odd turns: one barrier a turn
    __shared__ bool last;
    const int64_t b = blockIdx.x / (unsigned)A.groups;
    const int group = (int)(blockIdx.x - b * A.groups);
    const int lane = threadIdx.x & 63;
    const int n = drafts_of(A, b);

    bool ok = false;
    int x = -1;
    if (lane < n) {
        x = A.draft[b * A.K + lane];
        if (x >= 0 && x < A.V) {
            const double px = prob<T>(A.p, (b * (A.K + 1) + lane) * A.p_stride + x);
            const double qx = A.q ? prob<T>(A.q, (b * A.K + lane) * A.q_stride + x) : 1.0;
            ok = px >= 0.0 && qx >= 0.0 && (double)A.u_accept[b * A.K + lane] * qx < px;
        }
    }
    const int a = __ffsll((unsigned long long)~__ballot(ok)) - 1;  // n <= 63: some lane is false
    if (group == 0 && threadIdx.x < 64) {
        if (lane <= A.K && lane != a)
            A.tokens[b * (A.K + 1) + lane] = lane < a ? x : -1;
        if (lane == 0)
            A.accepted[b] = a;
    }

    const Draw d = draw_of(A, b, a, n);
    const E *const p = reinterpret_cast<const E *>(A.p) + d.p_row;
    const E *const q = d.q_row < 0 ? nullptr : reinterpret_cast<const E *>(A.q) + d.q_row;
    int turn = 0;
    for (int chunk = group; chunk < A.chunks; chunk += A.groups, turn++) {
        const int64_t base = (int64_t)chunk * kChunk;
        double sr = 0.0, sp = 0.0;
        if (base + kChunk <= A.V && (((uintptr_t)p | (uintptr_t)q) & 15) == 0) {
            EV pv[kPer / VEC], qv[kPer / VEC];
#pragma unroll
            for (int k = 0; k < kPer / VEC; k++) {
                pv[k] = *reinterpret_cast<const EV *>(p + base + (k * 256 + threadIdx.x) * VEC);
                qv[k] = q ? *reinterpret_cast<const EV *>(q + base + (k * 256 + threadIdx.x) * VEC) : EV(0);
            }
#pragma unroll
            for (int k = 0; k < kPer / VEC; k++)
#pragma unroll
                for (int e = 0; e < VEC; e++) {
                    const double pt = (double)(float)pv[k][e];
                    const bool out = base + (k * 256 + threadIdx.x) * VEC + e == d.out;
                    sr += out ? 0.0 : rest(pt, (double)(float)qv[k][e]);
                    sp += positive(pt);
                }
        } else {
            E pv[kPer], qv[kPer];
#pragma unroll
            for (int k = 0; k < kPer; k++) {
                const int64_t t = base + k * 256 + threadIdx.x;
                pv[k] = t < A.V ? p[t] : (E)0.0f;
                qv[k] = t < A.V && q ? q[t] : (E)0.0f;
            }
#pragma unroll
            for (int k = 0; k < kPer; k++) {
                const double pt = (double)(float)pv[k];
                sr += base + k * 256 + threadIdx.x == d.out ? 0.0 : rest(pt, (double)(float)qv[k]);
                sp += positive(pt);
            }
        }
        sr = wave_scan(sr);
        sp = wave_scan(sp);
        double2 (&w)[4] = lds[turn & 1];
        if (lane == 63)
            w[threadIdx.x >> 6] = make_double2(sr, sp);
        __syncthreads();
        if (threadIdx.x == 0)
            put_sum(A.sums + b * A.chunks + chunk, make_double2((w[0].x + w[1].x) + (w[2].x + w[3].x),
                                                                (w[0].y + w[1].y) + (w[2].y + w[3].y)));
    }
    if (threadIdx.x == 0) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the sums are at the device's scope
        last = arrive(A.arrivals + b * kLine, A.number) == (unsigned)A.groups;
        if (last)
            __hip_atomic_store(A.arrivals + b * kLine, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    if (last)
        choose<T>(A, b, n, a);
}

template <int T>
static int launch_verify(const VerifyArgs &A, int64_t B, hipStream_t s)
{
    hipLaunchKernelGGL((verify_kernel<T>), dim3((unsigned)(B * A.groups)), dim3(256), 0, s, A);
    return launch_status();
}

static int64_t verify_chunks(int64_t V) { return (V + kChunk - 1) / kChunk; }

// A number for a call, not zero, in the upper 44 bits: no two of 2^44 calls have the same.
static unsigned long long call_number()
{
    static std::atomic<unsigned long long> calls{0};
    unsigned long long n;
    do
        n = (calls.fetch_add(1, std::memory_order_relaxed) * 0x9E3779B97F4A7C15ull) << 20;
    while (n == 0);
    return n;
}

}  // namespace pn

using namespace pn;

extern "C" int64_t pn_verify_workspace_bytes(int64_t B, int64_t V)
{
    if (B < 0 || V < 1 || V >= (int64_t)1 << 30 || B > INT32_MAX / verify_chunks(V))
        return 0;
    return B * kLine * 8 + B * verify_chunks(V) * (int64_t)sizeof(double2);
}

extern "C" int pn_verify(int type, const void *p, int64_t p_stride, const void *q, int64_t q_stride,
                         const int32_t *draft, const int32_t *n_draft, const float *u_accept,
                         const float *u_sample, int64_t B, int64_t K, int64_t V, int32_t *tokens,
                         int32_t *accepted, void *workspace, int64_t workspace_bytes, void *stream)
{
    const int size = elem_bytes(type);
    if (size == 0)
        return PN_ERR_FORMAT;
    if (B < 0 || K < 0 || K > PN_VERIFY_MAX_DRAFTS || V < 1 || V >= (int64_t)1 << 30 ||
        B > INT32_MAX / verify_chunks(V))
        return PN_ERR_SHAPE;
    if (B == 0)
        return PN_OK;
    if (!p || !u_sample || !tokens || !accepted || !workspace || (K > 0 && (!draft || !u_accept)))
        return PN_ERR_NULL;
    if (!aligned(p, size) || !aligned(q, size) || !aligned(draft, 4) || !aligned(n_draft, 4) ||
        !aligned(u_accept, 4) || !aligned(u_sample, 4) || !aligned(tokens, 4) ||
        !aligned(accepted, 4) || !aligned(workspace, 16))
        return PN_ERR_ALIGN;
    if (workspace_bytes < pn_verify_workspace_bytes(B, V))
        return PN_ERR_WORKSPACE;
    const int st = check_device();
    if (st != PN_OK)
        return st;
    // enough workgroups to fill the memory pipe, few enough to arrive soon
    const int64_t chunks = verify_chunks(V);
    const int groups = (int)std::min<int64_t>(chunks, std::min<int64_t>(64, std::max<int64_t>(16, 1024 / B)));
    const VerifyArgs A{p, q, p_stride, q_stride, draft, n_draft, u_accept, u_sample, V, (int)K,
                       (int)chunks, groups, tokens, accepted, call_number(),
                       (unsigned long long *)workspace, (double2 *)((char *)workspace + B * kLine * 8)};
    hipStream_t s = (hipStream_t)stream;
    return type == PN_F32    ? launch_verify<PN_F32>(A, B, s)
           : type == PN_BF16 ? launch_verify<PN_BF16>(A, B, s)
                             : launch_verify<PN_F16>(A, B, s);
}
