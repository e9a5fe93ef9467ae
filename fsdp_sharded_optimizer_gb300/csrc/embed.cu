// embed.cu -- embedding lookup with scaling (zero_embed_forward) and its
// gradient by sorted tokens (zero_embed_backward).
//
//   out[t, :]    = scale * table[id_t, :]
//   dtable[v, :] = [old +] scale * sum over { t : id_t = v } of dout[t, :]
//
// The lookup is a copy with a scale: T*D elements read (fewer from HBM where
// ids repeat and the rows stay in the L2) and T*D written; HBM-bound, and for
// a few tokens latency-bound (one launch).
//
// The gradient has to add rows of dout that share an id.  Atomic adds would
// make the sum's order, and so its bits, change from run to run, would need
// an fp32 table, and would serialise on frequent tokens.  Here the tokens are
// put in the order of their ids (stable: by position where ids are equal), and
// the sorted list is cut into chunks of equal length, whatever rows they
// belong to, so that a token that makes up a tenth of the text costs no more
// than others.  A row whose tokens all lie in one chunk is finished there; one
// that goes across chunk borders leaves an fp32 partial sum per chunk, and
// those are added in order.  Every sum is fp32, in a fixed order, rounded once.
//
//   plan_kernel  each block owns a range of the vocabulary, counts its tokens
//                and puts them at their sorted places; rows without tokens
//                get their zeros here.
//   rows_kernel  the chunks' sums.
//   join_kernel  the rows that go across chunk borders.
//
// Read and written: T ids, T*D of dout, V*D of dtable (each row once), and
// 8*D bytes of partial sums per chunk at most.  HBM-bound.
#include "typed.cuh"
#include "zero_internal.h"

namespace zero {
namespace {

using dev::Bf16;

// ------------------------------------------------------------------ forward
constexpr int kLookupThreads = 256;
constexpr int kLookupUnroll = 4; // vectors a thread has in flight

template <int kVec, typename In, typename Out>
__global__ void __launch_bounds__(kLookupThreads)
lookup_kernel(const In* __restrict__ table, int64_t vocab, int64_t dim,
              const void* __restrict__ ids, int32_t id_type, int64_t n_tokens, float scale,
              Out* __restrict__ out)
{
    const uint32_t per_row = static_cast<uint32_t>(dim / kVec);
    const int64_t total = n_tokens * per_row;
    const int64_t base =
        static_cast<int64_t>(blockIdx.x) * (kLookupThreads * kLookupUnroll) + threadIdx.x;
    int64_t src[kLookupUnroll];
#pragma unroll
    for (int u = 0; u < kLookupUnroll; ++u) {
        const int64_t q = base + u * kLookupThreads;
        src[u] = -1;
        if (q < total) {
            const int64_t t = q / per_row;
            const int64_t id = dev::load_index(ids, id_type, t);
            if (id >= 0 && id < vocab) src[u] = id * dim + (q - t * per_row) * kVec;
        }
    }
    float x[kLookupUnroll][kVec];
#pragma unroll
    for (int u = 0; u < kLookupUnroll; ++u) {
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[u][e] = 0.0f;
        if (src[u] >= 0) dev::load_vec<kVec>(table + src[u], x[u]);
    }
#pragma unroll
    for (int u = 0; u < kLookupUnroll; ++u) {
        const int64_t q = base + u * kLookupThreads;
        if (q >= total) break;
        if (src[u] >= 0) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) x[u][e] *= scale;
        }
        dev::store_vec<kVec>(out + q * kVec, x[u]);
    }
}

template <typename In, typename Out>
int launch_lookup(const void* table, int64_t vocab, int64_t dim, const void* ids, int32_t id_type,
                  int64_t n_tokens, float scale, void* out, cudaStream_t stream)
{
    const bool wide = dim % 8 == 0 && aligned16(table) && aligned16(out);
    const int64_t total = n_tokens * (wide ? dim / 8 : dim);
    const int64_t per_block = kLookupThreads * kLookupUnroll;
    const int64_t blocks = (total + per_block - 1) / per_block;
    if (blocks > 0x7FFFFFFF) return ZERO_EINVAL;
    const auto* in = static_cast<const In*>(table);
    auto* o = static_cast<Out*>(out);
    if (wide)
        lookup_kernel<8, In, Out><<<static_cast<unsigned>(blocks), kLookupThreads, 0, stream>>>(
            in, vocab, dim, ids, id_type, n_tokens, scale, o);
    else
        lookup_kernel<1, In, Out><<<static_cast<unsigned>(blocks), kLookupThreads, 0, stream>>>(
            in, vocab, dim, ids, id_type, n_tokens, scale, o);
    return cuda_status(cudaGetLastError());
}

// ----------------------------------------------------------------- backward
constexpr int kPlanWarps = 32;
constexpr int kPlanThreads = kPlanWarps * 32;
constexpr int kPlanMaxBins = 1024; // rows of the vocabulary a block owns, at most
constexpr int kPlanBlocks = 152;   // wanted: one block per SM

struct PlanShape {
    int64_t bins, blocks;
    size_t smem;
};
PlanShape plan_shape(int64_t vocab)
{
    PlanShape s;
    s.bins = (vocab + kPlanBlocks - 1) / kPlanBlocks;
    if (s.bins > kPlanMaxBins) s.bins = kPlanMaxBins;
    s.blocks = (vocab + s.bins - 1) / s.bins;
    s.smem = static_cast<size_t>(s.bins) * (kPlanWarps + 1) * sizeof(uint32_t);
    return s;
}

// Sorted tokens per chunk.
constexpr int kChunk = 32;

struct EmbedScratch {
    int2* sorted;    // n_tokens: (token, id) in the order of (id, token)
    int32_t* starts; // vocab + 1: first sorted place of each row
    float* partial;  // chunks x 2 x dim: a chunk's first and last row, where they go on outside
    int64_t chunks, bytes;
};
EmbedScratch embed_scratch(void* base, int64_t n_tokens, int64_t vocab, int64_t dim)
{
    auto up = [](int64_t n) { return (n + 255) / 256 * 256; };
    EmbedScratch s;
    char* p = static_cast<char*>(base);
    int64_t at = 0;
    s.chunks = (n_tokens + kChunk - 1) / kChunk;
    s.sorted = reinterpret_cast<int2*>(p + at);
    at += up(n_tokens * 8);
    s.starts = reinterpret_cast<int32_t*>(p + at);
    at += up((vocab + 1) * 4);
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

// Sum over the block, valid in every thread.  `red` holds kPlanWarps + 1 words.
__device__ __forceinline__ uint32_t block_total(uint32_t x, uint32_t* red)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    uint32_t total = 0;
    for (int w = 0; w < kPlanWarps; ++w) total += red[w];
    return total;
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
            int2* __restrict__ sorted, int32_t* __restrict__ starts, char* __restrict__ dtable,
            int64_t row_bytes, int elem_bytes, int write_zeros)
{
    extern __shared__ uint32_t hist[]; // [kPlanWarps][bins], then row totals [bins]
    uint32_t* totals = hist + kPlanWarps * bins;
    __shared__ uint32_t red[kPlanWarps + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * bins;
    const int here = static_cast<int>(vocab - first < bins ? vocab - first : bins);
    for (int i = tid; i < kPlanWarps * bins; i += kPlanThreads) hist[i] = 0;
    __syncthreads();

    const int64_t run = ((n_tokens + kPlanWarps - 1) / kPlanWarps + 31) / 32 * 32;
    const int64_t lo = warp * run;
    const int64_t hi = lo + run < n_tokens ? lo + run : n_tokens;
    uint32_t* mine = hist + warp * bins;
    constexpr int kU = 4;
    uint32_t below = 0;
    for (int64_t i = lo + lane; i < hi; i += 32 * kU) {
        int64_t id[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) id[u] = i + 32 * u < hi ? static_cast<int64_t>(ids[i + 32 * u]) : -1;
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t b = id[u] - first;
            if (id[u] >= 0 && b < 0) ++below;
            if (b >= 0 && b < here && id[u] >= 0) atomicAdd(&mine[b], 1u);
        }
    }
    const uint32_t base = block_total(below, red);

    // totals of the rows, and each warp's place among the row's tokens
    for (int b = tid; b < here; b += kPlanThreads) {
        uint32_t sum = 0;
        for (int w = 0; w < kPlanWarps; ++w) {
            const uint32_t n = hist[w * bins + b];
            hist[w * bins + b] = sum;
            sum += n;
        }
        totals[b] = sum;
    }
    __syncthreads();
    // exclusive sum over the rows: kPlanMaxBins rows at most, one per thread
    const uint32_t mine_total = tid < here ? totals[tid] : 0;
    uint32_t incl = mine_total;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const uint32_t n = __shfl_up_sync(0xFFFFFFFFu, incl, off);
        if (lane >= off) incl += n;
    }
    __syncthreads();
    if (lane == 31) red[warp] = incl;
    __syncthreads();
    uint32_t before = 0;
    for (int w = 0; w < warp; ++w) before += red[w];
    const uint32_t start = base + before + incl - mine_total;
    if (tid < here) {
        starts[first + tid] = static_cast<int32_t>(start);
        if (first + tid == vocab - 1) starts[vocab] = static_cast<int32_t>(start + mine_total);
        for (int w = 0; w < kPlanWarps; ++w) hist[w * bins + tid] += start;
    }
    __syncthreads();

    for (int64_t i0 = lo; i0 < hi; i0 += 32 * kU) {
        int64_t id[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t i = i0 + 32 * u + lane;
            id[u] = i < hi ? static_cast<int64_t>(ids[i]) : -1;
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int64_t b = id[u] - first;
            const bool in = id[u] >= 0 && b >= 0 && b < here;
            const uint32_t any = __ballot_sync(0xFFFFFFFFu, in);
            if (any == 0) continue;
            uint32_t peers = 0, place = 0;
            if (in) {
                peers = __match_any_sync(any, static_cast<int>(b));
                place = mine[b];
            }
            __syncwarp();
            if (in) {
                const uint32_t rank = __popc(peers & ((1u << lane) - 1u));
                if (rank == 0) mine[b] = place + __popc(peers);
                sorted[place + rank] = make_int2(static_cast<int>(i0 + 32 * u + lane),
                                                 static_cast<int>(id[u]));
            }
            __syncwarp();
        }
    }
    if (!write_zeros) return;
    for (int b = warp; b < here; b += kPlanWarps)
        if (totals[b] == 0) warp_zero(dtable + (first + b) * row_bytes, row_bytes, elem_bytes, lane);
}

// One chunk of sorted tokens times one tile of columns; a thread holds kVec
// columns.  Loads of kRowsUnroll rows are issued together, whatever row
// borders lie between them.
constexpr int kRowsUnroll = 8;

template <int kVec, typename In, typename Out>
__global__ void __launch_bounds__(256)
rows_kernel(const In* __restrict__ dout, int64_t dim, const int2* __restrict__ sorted,
            const int32_t* __restrict__ starts, int64_t vocab, float scale, int accumulate,
            Out* __restrict__ dtable, float* __restrict__ partial)
{
    const int64_t n = starts[vocab];
    const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kChunk;
    if (c0 >= n) return;
    const int64_t c1 = c0 + kChunk < n ? c0 + kChunk : n;
    const int64_t col = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * kVec;
    if (col >= dim) return;
    int cur = sorted[c0].y;
    bool open = c0 > 0 && sorted[c0 - 1].y == cur; // begun in an earlier chunk
    float acc[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) acc[e] = 0.0f;

    auto finish = [&] {
        Out* o = dtable + static_cast<int64_t>(cur) * dim + col;
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
    };
    auto leave = [&](int slot) {
        dev::store_vec<kVec>(partial + (2 * static_cast<int64_t>(blockIdx.x) + slot) * dim + col,
                             acc);
    };

    for (int64_t i = c0; i < c1; i += kRowsUnroll) {
        float x[kRowsUnroll][kVec];
        int id[kRowsUnroll];
#pragma unroll
        for (int u = 0; u < kRowsUnroll; ++u) {
            if (i + u < c1) {
                const int2 s = sorted[i + u];
                id[u] = s.y;
                dev::load_vec<kVec>(dout + static_cast<int64_t>(s.x) * dim + col, x[u]);
            }
        }
#pragma unroll
        for (int u = 0; u < kRowsUnroll; ++u) {
            if (i + u < c1) {
                if (id[u] != cur) {
                    if (open)
                        leave(0);
                    else
                        finish();
                    open = false;
                    cur = id[u];
#pragma unroll
                    for (int e = 0; e < kVec; ++e) acc[e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < kVec; ++e) acc[e] += x[u][e];
            }
        }
    }
    if (open)
        leave(0);
    else if (c1 < n && sorted[c1].y == cur)
        leave(1);
    else
        finish();
}

// Rows that go across chunk borders: the block of the chunk in which a row
// begins adds that chunk's last partial and the first partials of the chunks
// up to the row's last token.  32 columns, kJoinSlices threads each; a slice
// adds a run of the chunks in order, the slices are added in order.
constexpr int kJoinSlices = 8;

template <typename Out>
__global__ void __launch_bounds__(32 * kJoinSlices)
join_kernel(int64_t dim, const int2* __restrict__ sorted, const int32_t* __restrict__ starts,
            int64_t vocab, float scale, int accumulate, Out* __restrict__ dtable,
            const float* __restrict__ partial)
{
    const int64_t n = starts[vocab];
    const int64_t c = blockIdx.x, c0 = c * kChunk, c1 = c0 + kChunk;
    if (c1 >= n) return;
    const int row = sorted[c1 - 1].y;
    if (sorted[c1].y != row) return;                 // ends here
    const int64_t begin = starts[row];
    if (begin < c0) return;                          // an earlier chunk's row
    const int64_t last = (starts[row + 1] - 1) / kChunk; // its last chunk
    const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
    const int64_t count = last - c; // first partials of chunks c + 1 .. last
    const int64_t per = (count + kJoinSlices - 1) / kJoinSlices;
    const int64_t lo = c + 1 + slice * per;
    const int64_t hi = lo + per < last + 1 ? lo + per : last + 1;
    __shared__ float sums[kJoinSlices][32];
    for (int64_t col0 = static_cast<int64_t>(blockIdx.y) * 32; col0 < dim;
         col0 += static_cast<int64_t>(gridDim.y) * 32) {
        const int64_t col = col0 + lane;
        float acc = 0.0f;
        if (col < dim) {
            if (slice == 0) acc = partial[(2 * c + 1) * dim + col];
#pragma unroll 4
            for (int64_t k = lo; k < hi; ++k) acc += partial[2 * k * dim + col];
        }
        __syncthreads();
        sums[slice][lane] = acc;
        __syncthreads();
        if (slice == 0 && col < dim) {
            float total = 0.0f;
#pragma unroll
            for (int s = 0; s < kJoinSlices; ++s) total += sums[s][lane];
            Out* o = dtable + static_cast<int64_t>(row) * dim + col;
            dev::store1(o, accumulate ? fmaf(scale, total, dev::load1(o)) : scale * total);
        }
    }
}

template <typename In, typename Out>
int launch_rows(const void* dout, int64_t dim, const EmbedScratch& s, int64_t vocab, float scale,
                int32_t accumulate, void* dtable, cudaStream_t stream)
{
    const bool wide = dim % 8 == 0 && aligned16(dout) && aligned16(dtable);
    const int64_t vecs = wide ? dim / 8 : dim;
    int threads = 256;
    if (vecs < threads) threads = static_cast<int>((vecs + 31) / 32 * 32);
    const dim3 grid(static_cast<unsigned>(s.chunks),
                    static_cast<unsigned>((vecs + threads - 1) / threads));
    const auto* in = static_cast<const In*>(dout);
    auto* out = static_cast<Out*>(dtable);
    if (wide)
        rows_kernel<8, In, Out><<<grid, threads, 0, stream>>>(in, dim, s.sorted, s.starts, vocab,
                                                              scale, accumulate, out, s.partial);
    else
        rows_kernel<1, In, Out><<<grid, threads, 0, stream>>>(in, dim, s.sorted, s.starts, vocab,
                                                              scale, accumulate, out, s.partial);
    const int rc = cuda_status(cudaGetLastError());
    if (rc != ZERO_OK || s.chunks < 2) return rc;
    const int64_t tiles = (dim + 31) / 32;
    const dim3 jgrid(static_cast<unsigned>(s.chunks - 1),
                     static_cast<unsigned>(tiles < 1024 ? tiles : 1024));
    join_kernel<Out><<<jgrid, 32 * kJoinSlices, 0, stream>>>(dim, s.sorted, s.starts, vocab, scale,
                                                             accumulate, out, s.partial);
    return cuda_status(cudaGetLastError());
}

constexpr int64_t kMaxTokens = int64_t(1) << 30; // places and starts are 32-bit
constexpr int64_t kMaxVocab = int64_t(1) << 30;
constexpr int64_t kMaxDim = int64_t(1) << 22;

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
    const int elem = type_bytes(dtable_type);
    const void* plan = id_type == ZERO_TYPE_I64
                           ? reinterpret_cast<const void*>(plan_kernel<int64_t>)
                           : reinterpret_cast<const void*>(plan_kernel<int32_t>);
    if (p.smem > 48 * 1024 &&
        cudaFuncSetAttribute(plan, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(p.smem)) != cudaSuccess)
        return ZERO_ECUDA;
    if (id_type == ZERO_TYPE_I64)
        plan_kernel<int64_t><<<static_cast<unsigned>(p.blocks), kPlanThreads, p.smem, stream>>>(
            static_cast<const int64_t*>(ids), n_tokens, vocab, static_cast<int>(p.bins), s.sorted,
            s.starts, static_cast<char*>(dtable), dim * elem, elem, !accumulate);
    else
        plan_kernel<int32_t><<<static_cast<unsigned>(p.blocks), kPlanThreads, p.smem, stream>>>(
            static_cast<const int32_t*>(ids), n_tokens, vocab, static_cast<int>(p.bins), s.sorted,
            s.starts, static_cast<char*>(dtable), dim * elem, elem, !accumulate);
    const int rc = cuda_status(cudaGetLastError());
    if (rc != ZERO_OK || n_tokens == 0) return rc;
    const float sc = static_cast<float>(scale);
    if (dout_type == ZERO_TYPE_BF16)
        return dtable_type == ZERO_TYPE_BF16
                   ? launch_rows<Bf16, Bf16>(dout, dim, s, vocab, sc, accumulate, dtable, stream)
                   : launch_rows<Bf16, float>(dout, dim, s, vocab, sc, accumulate, dtable, stream);
    return dtable_type == ZERO_TYPE_BF16
               ? launch_rows<float, Bf16>(dout, dim, s, vocab, sc, accumulate, dtable, stream)
               : launch_rows<float, float>(dout, dim, s, vocab, sc, accumulate, dtable, stream);
}
