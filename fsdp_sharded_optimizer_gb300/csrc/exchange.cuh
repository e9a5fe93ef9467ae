// exchange.cuh -- three words a turn, handed round among the blocks (ranks) of a
// cluster.
//
// They go by st.async, which counts its bytes on the receiver's mbarrier: a cluster
// barrier would have every thread wait for its own earlier stores to global memory
// first (the distillation of 2000 x 131072 bf16 on 4 ranks, then with 256 threads a
// block: 294 us with the barrier, 268 so).
// A rank that is in turn i has every rank's words of turn i-1, so all ranks have read
// those of turn i-2 and two sets of words in turn are enough.
//
// Every wait is limited.  A rank whose wait runs out is lost from then on: which words
// stand in its memory no longer goes by the turns, so it takes no further ones, and its
// caller has to leave NaN for this turn and all later ones.  It tells the others once,
// in the place of its next words (whatever they hold is then a NaN, too, for a rank
// that is still reading the set before), and they are lost when they read it.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace zero {
namespace dev {

constexpr int kMaxRanks = 8;

struct Words { // in shared memory
    float4 of[2][kMaxRanks]; // by the turn's parity: each rank's three words, and 1 where it is lost
    uint64_t arrived[2];     // mbarriers: all ranks' words of that parity are here
};

__device__ __forceinline__ uint32_t shared_at(const void* p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// By one thread; a cluster barrier has to follow before the first turn.
__device__ __forceinline__ void init_words(Words& words)
{
    for (int i = 0; i < 2; ++i)
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(shared_at(&words.arrived[i])) : "memory");
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void send_words(uint32_t words, uint32_t barrier, int to_rank, float a,
                                           float b, float c, uint32_t d)
{
    uint32_t there, there_barrier;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(words), "r"(to_rank));
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there_barrier) : "r"(barrier), "r"(to_rank));
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
                 ::"r"(there), "r"(__float_as_uint(a)), "r"(__float_as_uint(b)),
                 "r"(__float_as_uint(c)), "r"(d), "r"(there_barrier)
                 : "memory");
}
// Waits for the phase of a parity, a microsecond at a time; false after about a
// quarter of a second.
__device__ __forceinline__ bool wait_phase(uint32_t barrier, uint32_t phase)
{
    for (int i = 0; i < (1 << 18); ++i) {
        uint32_t done;
        asm volatile("{\n.reg .pred p;\n"
                     "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n"
                     "selp.u32 %0, 1, 0, p;\n}"
                     : "=r"(done)
                     : "r"(barrier), "r"(phase), "r"(1000u)
                     : "memory");
        if (done) return true;
    }
    return false;
}

// A thread's place in the turns; all threads of all ranks take every turn.
struct Turns {
    int parity = 0;    // of the next turn
    uint32_t phase = 0; // bit p: the phase that the mbarrier of parity p is in
    bool lost = false, told = false;

    // Hands a, b, c to every rank, and returns the ranks' words once they are here, to
    // be read before the thread's next turn.  Not valid where lost.
    __device__ __forceinline__ const float4* take(Words& words, int rank, int ranks, float a, float b,
                                                  float c)
    {
        const uint32_t barrier = shared_at(&words.arrived[parity]);
        const int tid = static_cast<int>(threadIdx.x);
        const float4* of = words.of[parity];
        if (tid == 0 && !lost)
            asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(barrier),
                         "r"(16 * ranks)
                         : "memory");
        if (tid < ranks && !told) {
            const float nan = __int_as_float(0x7FC00000);
            send_words(shared_at(&of[rank]), barrier, tid, lost ? nan : a, lost ? nan : b, lost ? nan : c,
                       lost ? 1u : 0u);
            told = lost;
        }
        if (!lost) {
            lost = !wait_phase(barrier, phase >> parity & 1);
            uint32_t gone = 0;
            for (int r = 0; r < ranks; ++r) gone |= __float_as_uint(of[r].w);
            lost = lost || gone != 0;
        }
        phase ^= 1u << parity;
        parity ^= 1;
        return of;
    }
};

} // namespace dev
} // namespace zero
