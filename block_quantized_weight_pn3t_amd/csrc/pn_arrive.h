// pn_arrive.h -- the last of the workgroups that share a piece of work: how they are counted and how
// what they left reaches the last one.
//
// Arrivals are counted in a word of the workspace, which nobody clears beforehand: its upper 44 bits
// hold the call's number, anything else there counts as zero arrivals, and the last one to arrive
// leaves zero, so a replayed graph finds it as the first run did. (An arrival takes about 30 ns of its
// word's cache line, one after another: a line a word, and not too many arrivals a word.) Which workgroup is
// last must change nothing in the result. What the workgroups leave are atomic stores and loads at the
// device's scope, as the eight XCDs' caches are not kept alike within a kernel: they pass those caches by,
// so all that is left to order is that a store is complete before the arrival is counted, by a wait, and
// that the loads come after the last arrival, by a barrier. (A release and an acquire at the device's scope
// promise the same in the language's terms, but the release writes the whole XCD's cache back.)
#pragma once

#include <atomic>

#include "pn_common.h"

namespace pn {

constexpr int kLine = 16;  // words of a cache line

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

// This workgroup's arrival, by one thread after its stores at the device's scope are complete: true in
// the last of `expected`, which leaves the word at zero.
__device__ __forceinline__ bool arrive_last(unsigned long long *word, unsigned long long number, unsigned expected)
{
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const bool last = arrive(word, number) == expected;
    if (last)
        __hip_atomic_store(word, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return last;
}

template <typename T>
__device__ __forceinline__ void put_shared(T *at, T v)
{
    __hip_atomic_store(at, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T get_shared(const T *at)
{
    return __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A number for a call, not zero, in the upper 44 bits: no two of 2^44 calls have the same.
inline unsigned long long call_number()
{
    static std::atomic<unsigned long long> calls{0};
    unsigned long long n;
    do
        n = (calls.fetch_add(1, std::memory_order_relaxed) * 0x9E3779B97F4A7C15ull) << 20;
    while (n == 0);
    return n;
}

}  // namespace pn
