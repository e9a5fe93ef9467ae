// embed.cu -- embedding lookup with scaling (zero_embed_forward) and its
// gradient by sorted tokens (zero_embed_backward).
//
//   out[t, :]    = scale * table[id_t, :]
//   dtable[v, :] = [old +] scale * sum over { t : id_t = v } of dout[t, :]
//
// The lookup is a copy with a scale: T*D elements read (fewer from HBM where
// ids repeat and the rows stay in the L2) and T*D written; HBM-bound, and for
// a few tokens bound by the launch (1.1 us on the device for one).
//
// The gradient has to add rows of dout that share an id.  Atomic adds would
// make the sum's order, and so its bits, change from run to run, would need
// an fp32 table, and would serialise on frequent tokens.  Here the tokens are
// put in the order of their ids (stable: by position where ids are equal), and
// the sorted list is cut into chunks of 16 or 32 tokens, whatever rows they
// belong to.  A chunk sums the rows that begin in it, a few tokens past its end
// where the last one's run on.  A frequent row, of more tokens than a chunk, is
// summed by all the chunks that it crosses, each leaving an fp32 partial sum,
// and those are added in order: a token that makes up a tenth of the text costs
// no more than others.  Every sum is fp32, in a fixed order, rounded once.
//
//   plan_kernel  each block owns a range of the vocabulary, counts its tokens
//                and puts them at their sorted places.
//   rows_kernel  the chunks' sums, and beside them the zeros of the rows
//                without tokens: reads and writes at once.
//   join_kernel  the frequent rows' sums over their chunks.
//
// Read and written: T ids, T*D of dout, V*D of dtable (each row once), and
// 8*D bytes of partial sums per chunk at most.  16384 x 4096 into 32000 rows takes
// 80 us for 396 MB, 262 MB of them written (4.9 TB/s): the plan 15 us, in which memory
// idles, the sums and zeros 62.  8192 x 768 into 50257 rows takes 29 us for 90 MB: the
// plan 11 us, the sums and zeros 18.5, whose 96-thread blocks of short rows wait for
// their loads at a third of the warps.  (Writes alone do not bound it: a fill of 262 MB
// takes 66 us, but the lookup, which reads as well, writes at 4.5 TB/s.)
#include "typed.cuh"
#include "zero_internal.h"

namespace zero {
namespace {

using dev::Bf16;

// ------------------------------------------------------------------ forward
constexpr int kLookupThreads = 256;
constexpr int kLookupUnroll = 4; // vectors a thread has in flight

// Block (t, y): the y-th stretch of token t's row; one id to a block.  HBM-bound:
// 16384 x 4096 bf16 takes 30.0 us, 6.0 TB/s; a thread per vector wherever it lies,
// with a division each, took 34.5, and rows of odd length (8000 x 1001) 22.0, not
// 13.1.
template <int kVec, typename In, typename Out>
__global__ void __launch_bounds__(kLookupThreads)
lookup_kernel(const In* __restrict__ table, int64_t vocab, int64_t dim,
              const void* __restrict__ ids, int32_t id_type, float scale, Out* __restrict__ out)
{
    const int64_t t = blockIdx.x;
    const int per_row = static_cast<int>(dim / kVec), threads = static_cast<int>(blockDim.x);
    const int first = static_cast<int>(blockIdx.y) * threads * kLookupUnroll + static_cast<int>(threadIdx.x);
    const int64_t id = dev::load_index(ids, id_type, t);
    const bool inside = id >= 0 && id < vocab;
    const In* row = table + (inside ? id : 0) * dim;
    Out* to = out + t * dim;
    float x[kLookupUnroll][kVec];
#pragma unroll
    for (int u = 0; u < kLookupUnroll; ++u) {
        const int v = first + u * threads;
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[u][e] = 0.0f;
        if (inside && v < per_row) dev::load_vec<kVec>(row + v * kVec, x[u]);
    }
#pragma unroll
    for (int u = 0; u < kLookupUnroll; ++u) {
        const int v = first + u * threads;
        if (v >= per_row) break;
        if (inside) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[u][e] *= scale;
        }
        dev::store_vec<kVec>(to + v * kVec, x[u]);
    }
}

template <typename In, typename Out>
int launch_lookup(const void* table, int64_t vocab, int64_t dim, const void* ids, int32_t id_type,
                  int64_t n_tokens, float scale, void* out, cudaStream_t stream)
{
    const bool wide = dim % 8 == 0 && aligned16(table) && aligned16(out);
    const int64_t per_row = wide ? dim / 8 : dim;
    // a row of up to 128 vectors takes one a thread, so that a warp's loads are whole
    int64_t threads = per_row <= 128 ? per_row : (per_row + kLookupUnroll - 1) / kLookupUnroll;
    threads = (threads + 31) / 32 * 32;
    if (threads > kLookupThreads) threads = kLookupThreads;
    const int64_t per_block = threads * kLookupUnroll;
    const dim3 grid(static_cast<unsigned>(n_tokens),
                    static_cast<unsigned>((per_row + per_block - 1) / per_block));
    const dim3 block(static_cast<unsigned>(threads));
    const auto* in = static_cast<const In*>(table);
    auto* o = static_cast<Out*>(out);
    if (wide)
        lookup_kernel<8, In, Out><<<grid, block, 0, stream>>>(in, vocab, dim, ids, id_type, scale, o);
    else
        lookup_kernel<1, In, Out><<<grid, block, 0, stream>>>(in, vocab, dim, ids, id_type, scale, o);
    return cuda_status(cudaGetLastError());
}

// ----------------------------------------------------------------- backward
constexpr int kPlanWarps = 32;
constexpr int kPlanThreads = kPlanWarps * 32;
constexpr int kPlanMaxBins = 1024; // rows of the vocabulary a block owns, at most
constexpr int kPlanBlocks = 152;   // wanted: one block per SM at most

constexpr size_t plan_smem(int64_t bins)
{
    return static_cast<size_t>(bins) * (kPlanWarps + 2) * sizeof(uint32_t);
}
struct PlanShape {
    int64_t bins, blocks;
    size_t smem;
};
PlanShape plan_shape(int64_t vocab)
{
    PlanShape s;
    s.bins = ((vocab + kPlanBlocks - 1) / kPlanBlocks + 31) / 32 * 32; // whole words of `empty`
    if (s.bins > kPlanMaxBins) s.bins = kPlanMaxBins;
    s.blocks = (vocab + s.bins - 1) / s.bins;
    s.smem = plan_smem(s.bins);
    return s;
}

// Sorted tokens per chunk; a row of more is frequent.  Depends on the sizes alone,
// so that the order of the sums does too.
// Measured (device time): 16384 x 4096 takes 84.5, 81.5 and 82.4 us with 16, 32
// and 64 a chunk, 8192 x 768 30.0, 32.3 and 40.0: few tokens want short chunks,
// whose rows are read one after the other.
constexpr int kMaxChunk = 32;
inline int chunk_size(int64_t n_tokens, int64_t dim)
{
    return n_tokens * dim < (int64_t(1) << 24) ? 16 : kMaxChunk;
}

struct EmbedScratch {
    int4* sorted;   // n_tokens: (token, id, first and end place of the id), by id, then token
    int32_t* count; // tokens whose id lies in the table
    uint32_t* empty; // a bit for each row of the table: no token has it
    float* partial; // chunks x 2 x dim: of the frequent row that a chunk begins in, and of the
                    // one that begins in it
    int per_chunk;
    int64_t chunks, bytes;
};
EmbedScratch embed_scratch(void* base, int64_t n_tokens, int64_t vocab, int64_t dim)
{
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    EmbedScratch s;
    char* p = static_cast<char*>(base);
    int64_t at = 0;
    s.per_chunk = chunk_size(n_tokens, dim);
    s.chunks = (n_tokens + s.per_chunk - 1) / s.per_chunk;
    s.sorted = reinterpret_cast<int4*>(p + at);
    at += up(n_tokens * 16);
    s.count = reinterpret_cast<int32_t*>(p + at);
    at += 256;
    s.empty = reinterpret_cast<uint32_t*>(p + at);
    at += up((vocab + 31) / 32 * 4);
    s.partial = reinterpret_cast<float*>(p + at);
    at += up(s.chunks * 2 * dim * 4);
    s.bytes = at;
    return s;
}

// Zeros n elements of `bytes` bytes each at p, by one warp: 16-byte stores
// over the aligned middle.
__device__ __forceinline__ void warp_zero(char* p, int64_t bytes, int elem_bytes, int lane)
{
    const int64_t to_aligned = (16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15;
    const int64_t head = to_aligned < bytes ? to_aligned : bytes;
    const int64_t body = (bytes - head) / 16;
    for (int64_t i = lane; i < body; i += 32)
        *reinterpret_cast<uint4*>(p + head + i * 16) = make_uint4(0, 0, 0, 0);
    auto zero_elem = [&](int64_t at) {
        if (elem_bytes == 2)
            *reinterpret_cast<uint16_t*>(p + at) = 0;
        else
            *reinterpret_cast<uint32_t*>(p + at) = 0;
    };
    for (int64_t at = lane * elem_bytes; at < head; at += 32 * elem_bytes) zero_elem(at);
    for (int64_t at = head + body * 16 + lane * elem_bytes; at < bytes; at += 32 * elem_bytes)
        zero_elem(at);
}

// An id as one word: those that are negative, or past 2^31, become 0xFFFFFFFF,
// which no row has.
__device__ __forceinline__ uint32_t id_word(int32_t id) { return id < 0 ? ~0u : static_cast<uint32_t>(id); }
__device__ __forceinline__ uint32_t id_word(int64_t id)
{
    return (id >> 31) != 0 ? ~0u : static_cast<uint32_t>(id);
}
__device__ __forceinline__ uint32_t warp_inclusive(uint32_t x, int lane)
{
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t n = __shfl_up_sync(0xFFFFFFFFu, x, off);
        if (lane >= off) x += n;
    }
    return x;
}

// A block owns rows [first, first + bins) of the vocabulary.  Warp w owns an
// equal run of the tokens.  First sweep: the warp counts its tokens of each
// row, and every thread counts the tokens of lower rows (all blocks read all
// ids; they stay in the L2).  Then hist[w][b] becomes the sorted place of warp
// w's first token of row b.  Second sweep: within 32 consecutive tokens, those
// of equal id find one another (match) and take consecutive places in lane
// order, so the order is stable and the same in every run; no float and no
// order-dependent atomic is involved.
template <typename Id>
__global__ void __launch_bounds__(kPlanThreads)
plan_kernel(const Id* __restrict__ ids, int64_t n_tokens, int64_t vocab, int bins,
            int4* __restrict__ sorted, int32_t* __restrict__ count, uint32_t* __restrict__ empty)
{
    extern __shared__ uint32_t hist[]; // [kPlanWarps][bins], then per row: first place, total
    uint32_t* firsts = hist + kPlanWarps * bins;
    uint32_t* totals = firsts + bins;
    __shared__ uint32_t red[2][kPlanWarps]; // of each warp: tokens of lower rows, of its rows
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * bins;
    const int here = static_cast<int>(vocab - first < bins ? vocab - first : bins);
    for (int i = tid; i < kPlanWarps * bins; i += kPlanThreads) hist[i] = 0;
    __syncthreads();

    // n_tokens <= 2^30: places and tokens are 32-bit
    const int tokens = static_cast<int>(n_tokens);
    const int run = ((tokens + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
    const int lo = warp * run;
    const int hi = tokens - lo < run ? tokens : lo + run; // at or below lo where nothing is left
    const uint32_t base_row = static_cast<uint32_t>(first), rows = static_cast<uint32_t>(here);
    uint32_t* mine = hist + warp * bins;
    constexpr int kU = 8;
    uint32_t below = 0;
    for (int i = lo + lane; i < hi; i += 32 * kU) {
        uint32_t id[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) id[u] = i + 32 * u < hi ? id_word(ids[i + 32 * u]) : ~0u;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            below += id[u] < base_row;
            if (id[u] - base_row < rows) atomicAdd(&mine[id[u] - base_row], 1u);
        }
    }
    below = __reduce_add_sync(0xFFFFFFFFu, below);
    if (lane == 0) red[0][warp] = below;
    __syncthreads();

    // the row's total, and its first place: kPlanMaxBins rows at most, one per thread
    uint32_t total = 0;
    if (tid < here) {
#pragma unroll
        for (int w = 0; w < kPlanWarps; ++w) total += hist[w * bins + tid];
    }
    const uint32_t incl = warp_inclusive(total, lane);
    if (lane == 31) red[1][warp] = incl;
    __syncthreads();
    const uint32_t base = __reduce_add_sync(0xFFFFFFFFu, red[0][lane]);
    const uint32_t before = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? red[1][lane] : 0u);
    const uint32_t start = base + before + incl - total;
    const uint32_t none = __ballot_sync(0xFFFFFFFFu, tid < here && total == 0);
    if (lane == 0 && tid < here) empty[(first + tid) / 32] = none;
    if (tid < here) {
        totals[tid] = total;
        firsts[tid] = start;
        if (first + tid == vocab - 1) *count = static_cast<int32_t>(start + total);
        if (total != 0) {
            uint32_t at = start;
#pragma unroll
            for (int w0 = 0; w0 < kPlanWarps; w0 += 8) {
                uint32_t n[8];
#pragma unroll
                for (int w = 0; w < 8; ++w) n[w] = hist[(w0 + w) * bins + tid];
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    hist[(w0 + w) * bins + tid] = at;
                    at += n[w];
                }
            }
        }
    }
    __syncthreads();

    for (int i0 = lo; i0 < hi; i0 += 32 * kU) {
        uint32_t id[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int i = i0 + 32 * u + lane;
            id[u] = i < hi ? id_word(ids[i]) : ~0u;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const uint32_t b = id[u] - base_row;
            const bool in = b < rows;
            const uint32_t any = __ballot_sync(0xFFFFFFFFu, in);
            if (any == 0) continue;
            uint32_t peers = 0, place = 0;
            if (in) {
                peers = __match_any_sync(any, b);
                place = mine[b];
            }
            __syncwarp();
            if (in) {
                const uint32_t rank = __popc(peers & ((1u << lane) - 1u));
                if (rank == 0) mine[b] = place + __popc(peers);
                const int at = static_cast<int>(firsts[b]);
                sorted[place + rank] = make_int4(i0 + 32 * u + lane, static_cast<int>(id[u]), at,
                                                 at + static_cast<int>(totals[b]));
            }
            __syncwarp();
        }
    }
}

// One chunk of sorted tokens times one tile of columns; a thread holds kVec
// columns.  The chunk's entries come to shared memory at once; then the loads of
// kRowsUnroll rows are issued together, whatever row borders lie between them.
constexpr int kRowsThreads = 256;
constexpr int kRowsUnroll = 8;
template <typename T, int kVec>
struct RawOf { // kVec elements as loaded
    T x;
};
template <typename T>
struct RawOf<T, 8> {
    dev::Raw8<T> x;
};
__device__ __forceinline__ void load_of(const Bf16* p, RawOf<Bf16, 8>& r) { dev::stream_raw8(p, r.x); }
__device__ __forceinline__ void load_of(const float* p, RawOf<float, 8>& r) { dev::stream_raw8(p, r.x); }
template <typename T>
__device__ __forceinline__ void load_of(const T* p, RawOf<T, 1>& r)
{
    r.x = *p;
}
template <typename T>
__device__ __forceinline__ void unpack_of(const RawOf<T, 8>& r, float (&x)[8])
{
    dev::unpack8(r.x, x);
}
template <typename T>
__device__ __forceinline__ void unpack_of(const RawOf<T, 1>& r, float (&x)[1])
{
    x[0] = dev::load1(&r.x);
}

template <int kVec, typename In, typename Out>
__global__ void __launch_bounds__(kRowsThreads, sizeof(In) == 2 ? 4 : 2)
rows_kernel(const In* __restrict__ dout, int64_t dim, int zero_blocks, int tiles, int per_chunk,
            const int4* __restrict__ sorted, const int32_t* __restrict__ count,
            const uint32_t* __restrict__ empty, float scale, int accumulate,
            Out* __restrict__ dtable, float* __restrict__ partial)
{
    __shared__ int4 entry[2 * kMaxChunk];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the zeros first: 16384 x 4096 takes 87.2 us with the chunks first, 87.5 in turn
    const int z = static_cast<int>(blockIdx.x), c = z - zero_blocks;
    if (z < zero_blocks) { // 32 rows of the table, a warp at one
        const uint32_t word = empty[z];
        for (int r = threadIdx.x >> 5; r < 32; r += static_cast<int>(blockDim.x) >> 5)
            if (word >> r & 1)
                warp_zero(reinterpret_cast<char*>(dtable + (static_cast<int64_t>(z) * 32 + r) * dim),
                          dim * sizeof(Out), sizeof(Out), threadIdx.x & 31);
        return;
    }
    const int n = *count;
    const int chunk = c / tiles, tile = c - chunk * tiles;
    const int c0 = chunk * per_chunk;
    if (c0 >= n) return;
    const int c1 = c0 + per_chunk < n ? c0 + per_chunk : n;
    for (int i = threadIdx.x; i < 2 * per_chunk; i += blockDim.x)
        if (c0 + i < n) entry[i] = sorted[c0 + i];
    __syncthreads();
    const int64_t col = (static_cast<int64_t>(tile) * blockDim.x + threadIdx.x) * kVec;
    if (col >= dim) return;
    // A row of no more than per_chunk tokens belongs to the chunk it begins in.
    auto frequent = [&](const int4& e) { return e.w - e.z > per_chunk; };
    const int4 head = entry[0], tail = entry[c1 - 1 - c0];
    const int begin = head.z < c0 && !frequent(head) ? head.w : c0;
    const int end = frequent(tail) ? c1 : tail.w;
    float acc[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) acc[e] = 0.0f;

    auto leave = [&](const int4& row) { // the sum of a row's tokens here
        if (frequent(row)) {
            const int slot = row.z < c0 ? 0 : 1;
            dev::store_vec<kVec>(
                partial + (2 * static_cast<int64_t>(chunk) + slot) * dim + col, acc);
        } else {
            Out* o = dtable + static_cast<int64_t>(row.y) * dim + col;
            float y[kVec];
            if (accumulate) {
                dev::load_vec<kVec>(o, y);
#pragma unroll
                for (int e = 0; e < kVec; ++e) y[e] = fmaf(scale, acc[e], y[e]);
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) y[e] = scale * acc[e];
            }
            dev::store_vec<kVec>(o, y);
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) acc[e] = 0.0f;
    };

    for (int i = begin; i < end; i += kRowsUnroll) {
        RawOf<In, kVec> raw[kRowsUnroll];
#pragma unroll
        for (int u = 0; u < kRowsUnroll; ++u)
            if (i + u < end)
                load_of(dout + static_cast<int64_t>(entry[i + u - c0].x) * dim + col, raw[u]);
#pragma unroll
        for (int u = 0; u < kRowsUnroll; ++u) {
            if (i + u < end) {
                float x[kVec];
                unpack_of(raw[u], x);
#pragma unroll
                for (int e = 0; e < kVec; ++e) acc[e] += x[e];
                const int4 row = entry[i + u - c0];
                if (i + u + 1 == row.w || i + u + 1 == end) leave(row);
            }
        }
    }
}

// The frequent rows: the chunk that one begins in holds its first partial sum,
// the chunks up to its last token the others.  Block x looks after the chunks
// x, x + gridDim.x, ...; kVec columns a lane, kJoinSlices threads for each: a
// slice adds a run of the chunks in order, the slices are added in order.
constexpr int kJoinSlices = 8, kJoinBlocks = 64;

template <int kVec, typename Out>
__global__ void __launch_bounds__(32 * kJoinSlices)
join_kernel(int64_t dim, int per_chunk, const int4* __restrict__ sorted, const int32_t* __restrict__ count,
            float scale, int accumulate, Out* __restrict__ dtable,
            const float* __restrict__ partial)
{
    __shared__ float sums[kJoinSlices][32][kVec];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int n = *count;
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t col = (static_cast<int64_t>(blockIdx.y) * 32 + lane) * kVec;
    // 32 chunks at a time are looked at, one by each lane
    for (int64_t c_base = blockIdx.x; c_base * per_chunk < n; c_base += 32 * static_cast<int64_t>(gridDim.x)) {
        const int64_t c_mine = c_base + static_cast<int64_t>(lane) * gridDim.x;
        int4 e = make_int4(0, 0, 0, 0);
        if ((c_mine + 1) * per_chunk <= n) e = sorted[(c_mine + 1) * per_chunk - 1]; // its last token
        uint32_t found = __ballot_sync(0xFFFFFFFFu, e.w - e.z > per_chunk && e.z >= c_mine * per_chunk);
        while (found) {
            const int who = __ffs(found) - 1;
            found &= found - 1;
            const int64_t c = c_base + static_cast<int64_t>(who) * gridDim.x;
            const int row = __shfl_sync(0xFFFFFFFFu, e.y, who);
            const int64_t last = (__shfl_sync(0xFFFFFFFFu, e.w, who) - 1) / per_chunk;
            const int64_t per = (last - c + kJoinSlices - 1) / kJoinSlices;
            const int64_t lo = c + 1 + slice * per;
            const int64_t hi = lo + per < last + 1 ? lo + per : last + 1;
            float acc[kVec], x[kVec];
#pragma unroll
            for (int v = 0; v < kVec; ++v) acc[v] = 0.0f;
            auto add = [&](const float* p) {
                if constexpr (kVec == 4) {
                    const float4 q = *reinterpret_cast<const float4*>(p);
                    x[0] = q.x, x[1] = q.y, x[2] = q.z, x[3] = q.w;
                } else {
                    x[0] = *p;
                }
#pragma unroll
                for (int v = 0; v < kVec; ++v) acc[v] += x[v];
            };
            if (col < dim) {
                if (slice == 0) add(partial + (2 * c + 1) * dim + col);
#pragma unroll 4
                for (int64_t k = lo; k < hi; ++k) add(partial + 2 * k * dim + col);
            }
            __syncthreads();
#pragma unroll
            for (int v = 0; v < kVec; ++v) sums[slice][lane][v] = acc[v];
            __syncthreads();
            if (slice == 0 && col < dim) {
                Out* o = dtable + static_cast<int64_t>(row) * dim + col;
#pragma unroll
                for (int v = 0; v < kVec; ++v) {
                    float total = 0.0f;
#pragma unroll
                    for (int s = 0; s < kJoinSlices; ++s) total += sums[s][lane][v];
                    dev::store1(o + v,
                                accumulate ? fmaf(scale, total, dev::load1(o + v)) : scale * total);
                }
            }
        }
    }
}

// A launch that may begin while the kernel before it on the stream drains; the
// kernel waits for that one's results itself.
template <typename... Params, typename... Given>
int launch_after(void (*kernel)(Params...), dim3 grid, dim3 block, cudaStream_t stream, Given... given)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(given)...));
}

template <typename In, typename Out>
int launch_rows(const void* dout, int64_t dim, int64_t vocab, const EmbedScratch& s, float scale,
                int32_t accumulate, void* dtable, cudaStream_t stream)
{
    const bool wide = dim % 8 == 0 && aligned16(dout) && aligned16(dtable);
    const int64_t vecs = wide ? dim / 8 : dim;
    int threads = kRowsThreads;
    if (vecs < threads) threads = static_cast<int>((vecs + 31) / 32 * 32);
    const int64_t tiles = (vecs + threads - 1) / threads;
    const int64_t zero_blocks = accumulate ? 0 : (vocab + 31) / 32;
    const int64_t blocks = zero_blocks + s.chunks * tiles;
    if (blocks == 0) return ZERO_OK;
    if (blocks > 0x7FFFFFFF) return ZERO_EINVAL;
    const dim3 grid(static_cast<unsigned>(blocks));
    const auto* in = static_cast<const In*>(dout);
    auto* out = static_cast<Out*>(dtable);
    const int rc =
        wide ? launch_after(rows_kernel<8, In, Out>, grid, dim3(threads), stream, in, dim,
                            zero_blocks, tiles, s.per_chunk, s.sorted, s.count, s.empty, scale, accumulate, out,
                            s.partial)
             : launch_after(rows_kernel<1, In, Out>, grid, dim3(threads), stream, in, dim,
                            zero_blocks, tiles, s.per_chunk, s.sorted, s.count, s.empty, scale, accumulate, out,
                            s.partial);
    if (rc != ZERO_OK || s.chunks < 2) return rc;
    const bool four = dim % 4 == 0;
    const int64_t strips = (dim + (four ? 127 : 31)) / (four ? 128 : 32);
    const dim3 jgrid(static_cast<unsigned>(s.chunks < kJoinBlocks ? s.chunks : kJoinBlocks),
                     static_cast<unsigned>(strips));
    return four ? launch_after(join_kernel<4, Out>, jgrid, dim3(32 * kJoinSlices), stream, dim,
                               s.per_chunk, s.sorted, s.count, scale, accumulate, out, s.partial)
                : launch_after(join_kernel<1, Out>, jgrid, dim3(32 * kJoinSlices), stream, dim,
                               s.per_chunk, s.sorted, s.count, scale, accumulate, out, s.partial);
}

constexpr int64_t kMaxTokens = int64_t(1) << 30; // places and starts are 32-bit
constexpr int64_t kMaxVocab = int64_t(1) << 30;
constexpr int64_t kMaxDim = int64_t(1) << 20;

bool embed_sizes_ok(int64_t vocab, int64_t dim, int64_t n_tokens)
{
    return vocab >= 1 && vocab <= kMaxVocab && dim >= 1 && dim <= kMaxDim && n_tokens >= 0 &&
           n_tokens <= kMaxTokens;
}

} // namespace
} // namespace zero

using namespace zero;

extern "C" int zero_embed_forward(const void* table, int32_t table_type, int64_t vocab,
                                  int64_t dim, const void* ids, int32_t id_type,
                                  int64_t n_tokens, double scale, void* out, int32_t out_type,
                                  cudaStream_t stream)
{
    if (!embed_sizes_ok(vocab, dim, n_tokens) || !float_type(table_type) ||
        !float_type(out_type) || !index_type(id_type))
        return ZERO_EINVAL;
    if (n_tokens == 0) return ZERO_OK;
    if (!table || !ids || !out) return ZERO_EINVAL;
    if (!aligned_to(table, type_bytes(table_type)) || !aligned_to(ids, type_bytes(id_type)) ||
        !aligned_to(out, type_bytes(out_type)))
        return ZERO_EALIGN;
    const float s = static_cast<float>(scale);
    if (table_type == ZERO_TYPE_BF16)
        return out_type == ZERO_TYPE_BF16
                   ? launch_lookup<Bf16, Bf16>(table, vocab, dim, ids, id_type, n_tokens, s, out,
                                               stream)
                   : launch_lookup<Bf16, float>(table, vocab, dim, ids, id_type, n_tokens, s, out,
                                                stream);
    return out_type == ZERO_TYPE_BF16
               ? launch_lookup<float, Bf16>(table, vocab, dim, ids, id_type, n_tokens, s, out,
                                            stream)
               : launch_lookup<float, float>(table, vocab, dim, ids, id_type, n_tokens, s, out,
                                             stream);
}

extern "C" int64_t zero_embed_scratch_bytes(int64_t n_tokens, int64_t vocab, int64_t dim)
{
    if (!embed_sizes_ok(vocab, dim, n_tokens)) return ZERO_EINVAL;
    return embed_scratch(nullptr, n_tokens, vocab, dim).bytes;
}

extern "C" int zero_embed_backward(const void* dout, int32_t dout_type, const void* ids,
                                   int32_t id_type, int64_t n_tokens, double scale, void* dtable,
                                   int32_t dtable_type, int64_t vocab, int64_t dim,
                                   int32_t accumulate, void* scratch, int64_t scratch_bytes,
                                   cudaStream_t stream)
{
    if (!embed_sizes_ok(vocab, dim, n_tokens) || !float_type(dout_type) ||
        !float_type(dtable_type) || !index_type(id_type) || !dtable || !scratch ||
        (accumulate != 0 && accumulate != 1))
        return ZERO_EINVAL;
    if (n_tokens > 0 && (!dout || !ids)) return ZERO_EINVAL;
    const EmbedScratch s = embed_scratch(scratch, n_tokens, vocab, dim);
    if (scratch_bytes < s.bytes) return ZERO_EINVAL;
    if (!aligned_to(dout, type_bytes(dout_type)) || !aligned_to(ids, type_bytes(id_type)) ||
        !aligned_to(dtable, type_bytes(dtable_type)) || !aligned16(scratch))
        return ZERO_EALIGN;
    if (n_tokens == 0 && accumulate) return ZERO_OK;

    const PlanShape p = plan_shape(vocab);
    const void* plan = id_type == ZERO_TYPE_I64
                           ? reinterpret_cast<const void*>(plan_kernel<int64_t>)
                           : reinterpret_cast<const void*>(plan_kernel<int32_t>);
    if (p.smem > 32 * 1024 && !allow_shared(plan, plan_smem(kPlanMaxBins))) // beside the static words
        return ZERO_ECUDA;
    const unsigned blocks = static_cast<unsigned>(p.blocks);
    const int bins = static_cast<int>(p.bins);
    if (id_type == ZERO_TYPE_I64)
        plan_kernel<int64_t><<<blocks, kPlanThreads, p.smem, stream>>>(
            static_cast<const int64_t*>(ids), n_tokens, vocab, bins, s.sorted, s.count, s.empty);
    else
        plan_kernel<int32_t><<<blocks, kPlanThreads, p.smem, stream>>>(
            static_cast<const int32_t*>(ids), n_tokens, vocab, bins, s.sorted, s.count, s.empty);
    const int rc = cuda_status(cudaGetLastError());
    if (rc != ZERO_OK) return rc;
    const float sc = static_cast<float>(scale);
    if (dout_type == ZERO_TYPE_BF16)
        return dtable_type == ZERO_TYPE_BF16
                   ? launch_rows<Bf16, Bf16>(dout, dim, vocab, s, sc, accumulate, dtable, stream)
                   : launch_rows<Bf16, float>(dout, dim, vocab, s, sc, accumulate, dtable, stream);
    return dtable_type == ZERO_TYPE_BF16
               ? launch_rows<float, Bf16>(dout, dim, vocab, s, sc, accumulate, dtable, stream)
               : launch_rows<float, float>(dout, dim, vocab, s, sc, accumulate, dtable, stream);
}
