// pn_logprobs.hip -- rows of logits as distributions: log probability and rank of a token, entropy, and
// the likeliest tokens, on gfx950.
//
// With m a row's maximum, d = x - m, l = sum e^(s d) and t = sum e^(s d) d (s the scale): log p = s d - log l
// and entropy = log l - s t / l, in which nothing cancels (log l >= 0 >= t). One pass: each lane keeps m, l and t
// of what it has seen and rescales them where m moves; partial results join likewise (t' = f (t + (m - m') l),
// f = e^(s (m - m'))).
//
// The likeliest tokens: a wave keeps its 64 best so far, one a lane, in falling order of a 64-bit key, the
// logit's bits in an order of whole numbers over the token's number inverted: equal logits fall by number and
// no two keys are equal. A batch of logits is looked at only where one passes the last that counts, which
// after the first batches is rare (about top / n of the logits at the n-th); then each lane offers its
// best, and few are put in one by one, many are sorted among the lanes and merged.
//
// Memory bound for long rows: 2047 of 248,320 bf16 171 us with the five likeliest (169 to 181 over several boxes, 5.6 to 6.0
// TB/s; a copy reaches 4.9, the exponentials and the rest would take about 150 by themselves). One row of fp32 13.6 us with 20,
// 8.5 with none, of which a launch and a first load are 5. Between one row and some hundred the lists are what is far from the
// floor: each wave begins one anew and raises its threshold by what it has seen itself (195 rows of 65,536 bf16 10.6 us with
// none, 19.2 with five, 23.8 with 20). A wave reads batches of 4 KB, one ahead; a row is shared by up to 64
// workgroups where there are few, and the last to arrive joins them (pn_arrive.h).
#include <float.h>

#include <algorithm>

#include "pn_arrive.h"
#include "pn_cache.h"
#include "pn_lanes.h"
#include "pn_launch.h"

namespace pn {

struct LogArgs {
    const void *logits;
    const int32_t *tokens;
    int64_t stride;
    int V, top, groups, batches;
    float scale, exp2_scale;  // of the logits; times log2(e)
    float *logprob, *entropy, *lse, *top_logprobs;
    int32_t *rank, *top_ids;
    u64 number;
    u64 *arrivals;  // [row][kLine]
    u64 *parts;     // [row][group][2]: m and l, t and count
    u64 *keys;      // [row][group][top]
};

// A row's (or a lane's) sums so far. m = -infinity: none. A NaN, or the difference of two infinities, stays
// in l from where it came up.
struct Sums {
    float m, l, t;
    int count;  // logits larger than the token's
};

__device__ __forceinline__ float greater(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, INFINITY); }

// From here on a maximum or minimum with a signalling NaN is the other operand, as with a quiet one. (As waves begin, with bit
// 9 of their mode register set, IEEE, it is a NaN, which the next maximum drops, and with it what came before.) In assembly,
// since the compiler takes the builtin for a write of memory.
__device__ __forceinline__ void pass_nan_by() { asm volatile("s_setreg_imm32_b32 hwreg(HW_REG_MODE, 9, 1), 0"); }

// The largest and the smallest of three, NaN aside after pass_nan_by(). (Left to itself the compiler quiets each operand
// first.)
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c)
{
    float r;
    asm("v_min3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// l and t relative to `from` as they are relative to `to`.
__device__ __forceinline__ void rescale(float &l, float &t, float from, float to, float exp2_scale)
{
    const float d = l > 0.0f ? from - to : 0.0f;
    const float f = __builtin_amdgcn_exp2f(d * exp2_scale);
    t = f > 0.0f ? f * __builtin_fmaf(d, l, t) : 0.0f;
    l = f * l;
}

__device__ __forceinline__ Sums join(Sums a, Sums b, float exp2_scale)
{
    const float m = greater(a.m, b.m);
    if (!(a.l == 0.0f))
        rescale(a.l, a.t, a.m, m, exp2_scale);
    if (!(b.l == 0.0f))
        rescale(b.l, b.t, b.m, m, exp2_scale);
    return Sums{m, a.l + b.l, a.t + b.t, a.count + b.count};
}

// The sums of all lanes, in every lane.
template <int MASK = 1>
__device__ __forceinline__ Sums over_lanes(Sums a, float exp2_scale)
{
    const auto other = [](auto v) { return __builtin_bit_cast(decltype(v), moved_by<MASK>(__builtin_bit_cast(uint32_t, v))); };
    a = join(a, Sums{other(a.m), other(a.l), other(a.t), other(a.count)}, exp2_scale);
    if constexpr (MASK < 32)
        return over_lanes<2 * MASK>(a, exp2_scale);
    else
        return a;
}

// A logit and its token as a key: larger logits first, then lower numbers; never 0.
__device__ __forceinline__ u64 key_of(float x, int token)
{
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);  // -0 as +0
    return (u64)(b >> 31 ? ~b : b | 0x80000000u) << 32 | (uint32_t)~token;
}
__device__ __forceinline__ float logit_of(u64 key)
{
    const uint32_t b = (uint32_t)(key >> 32);
    return __builtin_bit_cast(float, b >> 31 ? b & 0x7FFFFFFFu : ~b);
}
__device__ __forceinline__ int token_of(u64 key) { return (int)~(uint32_t)key; }

__device__ __forceinline__ u64 lane_key(u64 v, int lane)
{
    return (u64)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// The keys of this lane and of the one STRIDE away, the lower lane's first, in both lanes.
template <int STRIDE>
__device__ __forceinline__ void pair_of(u64 v, u64 &low, u64 &high)
{
    uint32_t l[2], h[2];
    const uint32_t w[2] = {(uint32_t)v, (uint32_t)(v >> 32)};
#pragma unroll
    for (int i = 0; i < 2; i++) {
        if constexpr (STRIDE == 32) {
            const auto p = __builtin_amdgcn_permlane32_swap(w[i], w[i], false, false);
            l[i] = p[0];
            h[i] = p[1];
        } else {
            const auto p = __builtin_amdgcn_permlane16_swap(w[i], w[i], false, false);
            l[i] = p[0];
            h[i] = p[1];
        }
    }
    low = (u64)l[1] << 32 | l[0];
    high = (u64)h[1] << 32 | h[0];
}
// One step of a bitonic network over the lanes: the larger or the smaller of the two that are STRIDE apart.
template <int STRIDE>
__device__ __forceinline__ u64 exchange(u64 v, bool larger)
{
    if constexpr (STRIDE >= 16) {
        u64 a, b;
        pair_of<STRIDE>(v, a, b);
        return (a > b) == larger ? a : b;
    } else {
        const u64 o = moved_by<STRIDE>(v);
        return (o > v) == larger ? o : v;
    }
}
template <int SIZE, int STRIDE>
__device__ __forceinline__ u64 network(u64 v, int lane)
{
    v = exchange<STRIDE>(v, ((lane & STRIDE) == 0) == ((lane & SIZE) == 0));
    if constexpr (STRIDE > 1)
        return network<SIZE, STRIDE / 2>(v, lane);
    else if constexpr (SIZE < 64)
        return network<SIZE * 2, SIZE>(v, lane);
    else
        return v;
}
// The lanes' keys in falling order.
__device__ __forceinline__ u64 sorted(u64 v, int lane) { return network<2, 1>(v, lane); }
// The 64 largest of two lists in falling order.
__device__ __forceinline__ u64 merged(u64 a, u64 b, int lane)
{
    const u64 r = moved_by<63>(b);
    return network<64, 32>(a > r ? a : r, lane);
}
// `key` put into the list (its last one falls out).
__device__ __forceinline__ u64 inserted(u64 list, u64 key, int lane)
{
    const int at = __popcll(__ballot(list > key));
    // wave_shr 1
    const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)list, 0x138, 0xF, 0xF, false);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(list >> 32), 0x138, 0xF, 0xF, false);
    return lane < at ? list : lane == at ? key : ((u64)hi << 32 | lo);
}

// A lane's part of a batch: 4 loads of VEC logits.
template <int T>
struct Batch {
    typedef typename Elem<T>::type E;
    static constexpr int VEC = 16 / sizeof(E), LOADS = 4, PER = VEC * LOADS, ALL = 64 * PER;
    typedef E EV __attribute__((ext_vector_type(VEC), aligned(sizeof(E))));  // rows of any alignment
    EV v[LOADS];
    // Logits from `base` on of a row of V (-infinity past its end).
    __device__ __forceinline__ void load(const E *row, int base, int V, int lane)
    {
#pragma unroll
        for (int i = 0; i < LOADS; i++) {
            const int at = base + i * 64 * VEC;
            if (at + 64 * VEC <= V) {
                // each line is read once (2047 rows of 248,320 bf16, 5 likeliest: 177 us, 187 by ordinary loads)
                v[i] = __builtin_nontemporal_load(reinterpret_cast<const EV *>(row + at + lane * VEC));
            } else {
#pragma unroll
                for (int j = 0; j < VEC; j++)
                    v[i][j] = at + lane * VEC + j < V ? row[at + lane * VEC + j] : (E)-INFINITY;
            }
        }
    }
};

// Puts what passes `thr` of a batch whose first logit of this lane is token `first` into the list; m is the lane's
// largest.
template <int T>
__device__ __forceinline__ void take(const float (&x)[Batch<T>::PER], float m, int first, int top, int lane, u64 &list,
                                     float &thr)
{
    constexpr int VEC = Batch<T>::VEC, PER = Batch<T>::PER;
    const auto token = [&](int j) { return first + j / VEC * 64 * VEC + j % VEC; };
    if (__popcll(__ballot(m > thr)) <= 4) {
        // few lanes: each logit that passes is put in by itself
#pragma unroll
        for (int j = 0; j < PER; j++) {
            u64 offers = __ballot(x[j] > thr);
            if (offers) {
                const u64 key = key_of(x[j], token(j));
                for (; offers; offers &= offers - 1)
                    list = inserted(list, lane_key(key, __ffsll(offers) - 1), lane);
            }
        }
    } else {
        // each lane offers its best, and those that pass are sorted among the lanes and merged, until none passes
        uint32_t left = 0;
#pragma unroll
        for (int j = 0; j < PER; j++)
            left |= x[j] > thr ? 1u << j : 0u;
        while (__any(left != 0)) {
            float best = -INFINITY;
            int at = 0;
#pragma unroll
            for (int j = 0; j < PER; j++)
                if ((left >> j & 1) && x[j] > best) {
                    best = x[j];
                    at = j;
                }
            const u64 key = key_of(best, token(at));
            const bool in = left != 0 && key > lane_key(list, top - 1);
            left = in ? left & ~(1u << at) : 0;
            u64 offers = __ballot(in);
            if (__popcll(offers) > 8) {
                const u64 fresh = sorted(in ? key : 0, lane);
                list = lane_key(list, 0) ? merged(list, fresh, lane) : fresh;
            } else {
                for (; offers; offers &= offers - 1)
                    list = inserted(list, lane_key(key, __ffsll(offers) - 1), lane);
            }
        }
    }
    const u64 last = lane_key(list, top - 1);
    thr = last ? logit_of(last) : -INFINITY;
}

// A row's outputs by one wave, from its sums and its list.
__device__ __forceinline__ void write_row(const LogArgs &A, int64_t row, Sums a, u64 list, int lane, float token_logit,
                                          bool has_token)
{
    const float nan = __builtin_nanf("");
    const bool bad = !(a.l < INFINITY);  // a NaN or +infinity
    const float log_l = logf(a.l);
    const auto log_p = [&](float x) {
        float d = A.scale * (x - a.m);
        if (!(d > -INFINITY))  // a difference that passes fp32 comes back where the scale is below one
            d = (float)((double)A.scale * ((double)x - (double)a.m));
        return bad || a.l == 0.0f ? nan : d - log_l;
    };
    if (lane == 0) {
        if (A.logprob)
            A.logprob[row] = has_token ? log_p(token_logit) : 0.0f;
        if (A.rank)
            A.rank[row] = has_token ? a.count : -1;
        if (A.entropy)
            A.entropy[row] = bad || a.l == 0.0f ? nan : log_l - A.scale * (a.t / a.l);
        if (A.lse)
            A.lse[row] = bad ? nan : a.l == 0.0f ? -INFINITY : __builtin_fmaf(A.scale, a.m, log_l);
    }
    if (lane < A.top) {
        A.top_ids[row * A.top + lane] = list ? token_of(list) : -1;
        A.top_logprobs[row * A.top + lane] = bad ? nan : list ? log_p(logit_of(list)) : -INFINITY;
    }
}

// The lists of a workgroup's waves into the first one's, by twos, behind one barrier at least.
template <int WAVES>
__device__ __forceinline__ u64 over_waves(u64 list, u64 (&lds)[WAVES][64], int wave, int lane, int top)
{
    if (top == 0) {
        __syncthreads();
        return 0;
    }
#pragma unroll
    for (int n = WAVES / 2; n > 0; n /= 2) {
        if (wave >= n && wave < 2 * n)
            lds[wave][lane] = list;
        __syncthreads();
        if (wave < n)
            list = merged(list, lds[wave + n][lane], lane);
    }
    return list;
}

template <int T, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, 4) logprobs_kernel(LogArgs A)
{
    typedef Batch<T> B;
    typedef typename B::E E;
    constexpr bool SHARED = WAVES < 16;  // whether rows can have several workgroups (log_groups)
    __shared__ Sums lds_sums[WAVES];
    __shared__ u64 lds_list[1 + SHARED][WAVES][64];
    __shared__ bool last;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t row = blockIdx.x / (unsigned)A.groups;
    const int group = (int)(blockIdx.x - row * A.groups);
    const E *const x_row = reinterpret_cast<const E *>(A.logits) + row * A.stride;

    int batch = group * WAVES + wave;
    B next;
    if (batch < A.batches)
        next.load(x_row, batch * B::ALL, A.V, lane);
    const int token = A.tokens ? A.tokens[row] : -1;
    const bool has_token = token >= 0 && token < A.V;
    const float token_logit = has_token ? (float)x_row[token] : INFINITY;
    pass_nan_by();

    Sums a{-INFINITY, 0.0f, 0.0f, 0};
    float ref = 0.0f;  // what l and t are relative to: m, or anything while they are zero
    u64 list = 0;
    float thr = A.top > 0 ? -INFINITY : INFINITY;
    while (batch < A.batches) {
        const int first = batch * B::ALL + lane * B::VEC;
        const B now = next;
        batch += A.groups * WAVES;
        if (batch < A.batches)
            next.load(x_row, batch * B::ALL, A.V, lane);
        float x[B::PER];
#pragma unroll
        for (int j = 0; j < B::PER; j++)
            x[j] = (float)now.v[j / B::VEC][j % B::VEC];
        float m = -INFINITY, low = INFINITY;
#pragma unroll
        for (int j = 0; j < B::PER; j += 2) {
            m = max3(m, x[j], x[j + 1]);
            low = min3(low, x[j], x[j + 1]);
        }
        if (__any(m > thr))
            take<T>(x, m, first, A.top, lane, list, thr);
        if (__any(m > token_logit))
#pragma unroll
            for (int j = 0; j < B::PER; j++)
                a.count += x[j] > token_logit;
        m = greater(a.m, m);
        if (m > a.m) {
            rescale(a.l, a.t, ref, m, A.exp2_scale);
            a.m = ref = m;
        }
        // e is 0 where d is -infinity, and the product with it must be too
        const auto add = [&](auto masked) {
#pragma unroll
            for (int j = 0; j < B::PER; j++) {
                const float d = x[j] - ref, e = __builtin_amdgcn_exp2f(d * A.exp2_scale);
                a.l += e;
                a.t = __builtin_fmaf(e, masked.value ? greater(d, -FLT_MAX) : d, a.t);
            }
        };
        if (__any(low - ref == -INFINITY))
            add(std::true_type());
        else
            add(std::false_type());
    }
    a = over_lanes(a, A.exp2_scale);

    // the workgroup's waves into the first
    if (lane == 0)
        lds_sums[wave] = a;
    list = over_waves<WAVES>(list, lds_list[0], wave, lane, A.top);
    if (wave == 0) {
        a = lane < WAVES ? lds_sums[lane] : Sums{-INFINITY, 0.0f, 0.0f, 0};
        a = over_lanes(a, A.exp2_scale);
        if (!SHARED || A.groups == 1)
            write_row(A, row, a, list, lane, token_logit, has_token);
    }
    if (!SHARED || A.groups == 1)
        return;
    if (wave == 0) {
        const int64_t at = row * A.groups + group;
        if (lane == 0) {
            put_shared(A.parts + 2 * at, (u64)__builtin_bit_cast(uint32_t, a.l) << 32 | __builtin_bit_cast(uint32_t, a.m));
            put_shared(A.parts + 2 * at + 1, (u64)(uint32_t)a.count << 32 | __builtin_bit_cast(uint32_t, a.t));
        }
        if (lane < A.top)
            put_shared(A.keys + at * A.top + lane, list);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // every lane's stores
        if (lane == 0)
            last = arrive_last(A.arrivals + row * kLine, A.number, (unsigned)A.groups);
    }
    __syncthreads();
    if (!last)
        return;
    // the groups' lists dealt to the waves, read at once, merged by twos
    constexpr int EACH = 64 / WAVES;
    u64 in[EACH];
#pragma unroll
    for (int i = 0; i < EACH; i++) {
        const int g = wave + WAVES * i;
        in[i] = g < A.groups && lane < A.top ? get_shared(A.keys + (row * A.groups + g) * A.top + lane) : 0;
    }
    a = Sums{-INFINITY, 0.0f, 0.0f, 0};
    if (wave == 0 && lane < A.groups) {
        const u64 *const p = A.parts + 2 * (row * A.groups + lane);
        const u64 u = get_shared(p), v = get_shared(p + 1);
        a = Sums{__builtin_bit_cast(float, (uint32_t)u), __builtin_bit_cast(float, (uint32_t)(u >> 32)),
                 __builtin_bit_cast(float, (uint32_t)v), (int)(v >> 32)};
    }
#pragma unroll
    for (int n = EACH / 2; n > 0; n /= 2)
        if (A.groups > WAVES * n)
#pragma unroll
            for (int i = 0; i < n; i++)
                in[i] = merged(in[i], in[i + n], lane);
    list = over_waves<WAVES>(in[0], lds_list[SHARED], wave, lane, A.top);
    if (wave == 0)
        write_row(A, row, over_lanes(a, A.exp2_scale), list, lane, token_logit, has_token);
}

// A batch has 1024 logits of four bytes or 2048 of two.
static int log_batches(int type, int64_t V)
{
    const int all = type == PN_F32 ? Batch<PN_F32>::ALL : Batch<PN_BF16>::ALL;
    return (int)((V + all - 1) / all);
}

// Waves of a workgroup and workgroups of a row.
// Up to 512 rows: workgroups of eight waves, which a CU holds two of, and as many a row as the machine has CUs for; more
// begin more lists anew, and a second round of them costs the first one's time again. 195 rows of 65,536 bf16, 5
// likeliest: 20.0 us by one a row, 23.6 by two, 33.8 by two of 16 waves; 48 rows of 248,320: 20.6 by five a row, 23.3 by
// ten, 23.8 by five of 16 waves, 24.6 by five of four; one row of 248,320 fp32, 20 likeliest: 13.4, by 16 waves 15.6.
// A row of nine to 16 batches: one workgroup of 16 waves, which spares the hand-over (one row of 20,000 bf16: 5.8 us, 7.4
// by two of eight).
// More than 512 rows: one of four waves each, which a CU holds four of (1000 rows of 65,536 bf16, 5 likeliest: 38.4 us,
// 47.4 by eight waves; 511 rows: 27.6 by eight, 26.9 by four, 30.7 by two of four a row).
// 257 to 341 long rows: three of four waves each, as the second workgroups of eight waves would fall to few CUs (300 rows
// of 248,320 bf16, 5 likeliest: 48.7 us, 56.8 by eight waves; of 65,536 26.2 and 26.3, of 20,000 17.4 and 15.7).
static int log_waves(int64_t R, int batches)
{
    if (R > 512 || (R > 256 && R <= 341 && batches > 64))
        return 4;
    return R <= 256 && batches > 8 && batches <= 16 ? 16 : 8;
}
static int log_groups(int64_t R, int batches)
{
    const int waves = log_waves(R, batches);
    return (int)std::max<int64_t>(1, std::min<int64_t>({64, (batches + waves - 1) / waves, (waves == 4 ? 1024 : 256) / R}));
}

// A's rows from `first` on, of a workgroup each.
template <int T>
static LogArgs rows_from(LogArgs A, int64_t first)
{
    const auto from = [first](auto *p, int64_t stride) { return p ? p + first * stride : p; };
    A.logits = from((const typename Elem<T>::type *)A.logits, A.stride);
    A.tokens = from(A.tokens, 1);
    A.logprob = from(A.logprob, 1);
    A.rank = from(A.rank, 1);
    A.entropy = from(A.entropy, 1);
    A.lse = from(A.lse, 1);
    A.top_ids = from(A.top_ids, A.top);
    A.top_logprobs = from(A.top_logprobs, A.top);
    return A;
}

template <int T>
static int launch_log(LogArgs A, int64_t R, hipStream_t s)
{
    const int waves = log_waves(R, A.batches);
    const int64_t most = launch_most(64 * waves);  // rows share workgroups where there are far fewer
    for (;; A = rows_from<T>(A, most), R -= most) {
        const dim3 grid((unsigned)(std::min(R, most) * A.groups));
        if (waves == 16)
            hipLaunchKernelGGL((logprobs_kernel<T, 16>), grid, dim3(1024), 0, s, A);
        else if (waves == 8)
            hipLaunchKernelGGL((logprobs_kernel<T, 8>), grid, dim3(512), 0, s, A);
        else
            hipLaunchKernelGGL((logprobs_kernel<T, 4>), grid, dim3(256), 0, s, A);
        if (R <= most)
            return launch_status();
    }
}

static bool logits_fit(int64_t R, int64_t V, int top)
{
    return R >= 0 && R <= INT32_MAX / 64 && V >= 1 && V < (int64_t)1 << 30 && top >= 0 && top <= PN_LOGPROBS_MAX_TOP;
}

// Scales with which the sum of e^(s d) d stays within fp32: e^(s d) |d| is at most 0.37 / s and, where it is not zero, |d| at
// most 128 / s, which V times are 2^128 at most. (A d that passes fp32 then has e^(s d) = 0, as it should.)
static bool scale_fits(float scale, int64_t V) { return scale >= (float)V * 0x1p-121f && scale <= FLT_MAX; }

}  // namespace pn

using namespace pn;

extern "C" int64_t pn_logprobs_workspace_bytes(int64_t R, int64_t V, int top)
{
    if (!logits_fit(R, V, top) || R == 0)
        return 0;
    // as many shares of rows as log_groups deals at most, of the type that has more batches: enough for fewer rows too
    const int64_t shares = std::min(R * std::min(64, (log_batches(PN_F32, V) + 3) / 4), std::max<int64_t>(R, 1024));
    return R * kLine * 8 + shares * (2 + top) * 8;
}

extern "C" int pn_logprobs(const pn_logprobs_args *a, void *workspace, int64_t workspace_bytes, void *stream)
{
    if (!a)
        return PN_ERR_NULL;
    const int size = elem_bytes(a->type);
    if (size == 0)
        return PN_ERR_FORMAT;
    if (!logits_fit(a->R, a->V, a->top) || !scale_fits(a->scale, a->V))
        return PN_ERR_SHAPE;
    if (a->R == 0)
        return PN_OK;
    if (!a->logits || !workspace || ((a->logprob || a->rank) && !a->tokens) || (a->top > 0 && (!a->top_ids || !a->top_logprobs)))
        return PN_ERR_NULL;
    if (!aligned(a->logits, size) || !aligned(a->tokens, 4) || !aligned(a->logprob, 4) || !aligned(a->rank, 4) ||
        !aligned(a->entropy, 4) || !aligned(a->lse, 4) || !aligned(a->top_ids, 4) || !aligned(a->top_logprobs, 4))
        return PN_ERR_ALIGN;
    if (!aligned(workspace, 16))
        return PN_ERR_ALIGN;
    if (workspace_bytes < pn_logprobs_workspace_bytes(a->R, a->V, a->top))
        return PN_ERR_WORKSPACE;
    const int st = check_device();
    if (st != PN_OK)
        return st;
    LogArgs A = {};
    A.logits = a->logits;
    A.tokens = a->tokens;
    A.stride = a->stride;
    A.V = (int)a->V;
    A.top = a->top;
    A.batches = log_batches(a->type, a->V);
    A.groups = log_groups(a->R, A.batches);
    A.scale = a->scale;
    A.exp2_scale = (float)std::min((double)a->scale * 1.4426950408889634, (double)FLT_MAX);
    A.logprob = a->logprob;
    A.entropy = a->entropy;
    A.lse = a->lse;
    A.top_logprobs = a->top_logprobs;
    A.rank = a->rank;
    A.top_ids = a->top_ids;
    A.number = call_number();
    A.arrivals = (u64 *)workspace;
    A.parts = A.arrivals + a->R * kLine;
    A.keys = A.parts + a->R * A.groups * 2;
    hipStream_t s = (hipStream_t)stream;
    return a->type == PN_F32    ? launch_log<PN_F32>(A, a->R, s)
           : a->type == PN_BF16 ? launch_log<PN_BF16>(A, a->R, s)
                                : launch_log<PN_F16>(A, a->R, s);
}
