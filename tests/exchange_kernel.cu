// A cluster of `ranks` blocks that takes `turns` turns of exchange.cuh, with rank
// `late` two seconds late for turn `at` (none where late is negative): a wait of the
// others runs out.  out[turn][rank][thread]: the sum of all words, NaN where lost.
#include "exchange.cuh"

using namespace zero::dev;
constexpr int kThreads = 64;

__global__ void __launch_bounds__(kThreads) turns_kernel(int ranks, int turns, int late, int at, float* out)
{
    __shared__ Words words;
    const int tid = static_cast<int>(threadIdx.x), rank = static_cast<int>(blockIdx.x);
    if (tid == 0) init_words(words);
    __syncthreads();
    cluster_barrier();
    Turns mine;
    for (int i = 0; i < turns; ++i) {
        if (rank == late && i == at && tid == 0) {
            unsigned long long from, now;
            asm volatile("mov.u64 %0, %globaltimer;" : "=l"(from));
            for (int k = 0; k < 20000; ++k) {
                __nanosleep(1000000);
                asm volatile("mov.u64 %0, %globaltimer;" : "=l"(now));
                if (now - from > 2000000000ull) break;
            }
        }
        __syncthreads();
        const float4* of = mine.take(words, rank, ranks, 100.0f * (i % 64) + rank, static_cast<float>(i % 7),
                                     static_cast<float>(rank));
        float sum = mine.lost ? __int_as_float(0x7FC00000) : 0.0f;
        for (int r = 0; r < ranks; ++r) sum += of[r].x + of[r].y + of[r].z;
        out[(static_cast<long long>(i) * ranks + rank) * kThreads + tid] = sum;
    }
    cluster_barrier();
}

extern "C" int run_turns(int ranks, int turns, int late, int at, float* out, cudaStream_t stream)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(ranks);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return static_cast<int>(cudaLaunchKernelEx(&cfg, turns_kernel, ranks, turns, late, at, out));
}
