// relpos.cu -- the learned relative position bias by buckets
// (zero_relpos_forward) and the gradient of its table (zero_relpos_backward).
//
//   out[b, h, i, j] = scores[b, h, i, j] + table[bucket(j - i - start_b), h]
//   dtable[v, h]    = sum of dout[b, h, i, j] over the places with bucket v
//
// The buckets of one direction are the distances 0, 1, .., half - 1 and then
// parts of equal length on a logarithmic scale up to max_distance.  Where they
// begin (Borders) is found on the host in whole numbers, so that no rounding of a
// logarithm moves a distance into another bucket.  A bucket is an interval of
// the distance d = j - i - start, and d is constant along the diagonals.
//
// Both kernels take rows of 16-byte vectors aligned in memory, whatever the
// row's alignment: vector u of row i covers the columns 8u - lead .. 8u - lead + 7,
// where lead is how far the row starts behind such a boundary.
//
// Forward: each block lays out the bias by distance in shared memory once (the
// distances beyond the last border are one value), then streams its rows.
//
// Backward: no place needs its bucket.  A thread owns a slot, a diagonal of
// vectors: going down by eight rows its vector moves by one, so the 15 diagonals
// on which the elements of its vectors lie stay the same, and their sums stay in
// registers: one addition a place.  The sums of diagonals are added up by bucket
// at the end, the blocks' sums by a second kernel, in a fixed order.
//
// What bounds them: HBM.  Forward 32 x 2048 x 2048 bf16, the bias alone: 41 us, 6.6 TB/s; added
// to 8 x 12 x 1024 x 1024 scores 66 us, 6.1 TB/s, with a causal mask and padding 43 us, 4.8 TB/s
// (rows of unequal length, and a third of the issue slots).  Backward 4 x 32 x 2048 x 2048 bf16:
// 175 us, 6.1 TB/s; odd rows 2047 x 2047 234 us, 4.6 TB/s (the phase of a row is known only when
// it is loaded).  16 x 12 x 333 x 333, lengths down to half: 34 us, 0.7 TB/s: instructions, as
// nearly every row of a band has an end in it, and 576 unequal blocks on 456 places.
#include <algorithm>
#include <cmath>

#include "typed.cuh"
#include "zero_internal.h"

namespace zero {
namespace {

using dev::Bf16;
using dev::Raw8;

constexpr int kMaxBuckets = 512;
constexpr int64_t kMaxDistance = 8192;
constexpr int64_t kMaxLen = int64_t(1) << 24;
constexpr int64_t kMaxStride = int64_t(1) << 30;
constexpr int64_t kMaxStart = int64_t(1) << 40;

// Where the buckets of one direction begin: ascending distances, the first is 0.
struct Borders {
    int32_t n;    // buckets of one direction
    int32_t both; // 1: later keys have buckets of their own, after the others
    int16_t at[kMaxBuckets];
};

struct Geometry {
    int64_t out_plane, in_plane; // elements from one (b, h) to the next
    int64_t out_stride, in_stride;
    int64_t start;
    const int32_t *starts, *q_lengths, *k_lengths;
    int32_t batch, heads, q_len, k_len, causal;
};

__device__ __forceinline__ int64_t start_of(const Geometry& G, int b)
{
    return G.starts ? G.starts[b] : G.start;
}
__device__ __forceinline__ int length_of(const int32_t* lengths, int b, int most)
{
    if (!lengths) return most;
    const int n = lengths[b];
    return n < 0 ? 0 : n < most ? n : most;
}

// ------------------------------------------------------------------ forward
constexpr int kThreads = 256;

// The bias by distance in shared memory: place k stands for the distance k - 8 - last,
// held within [-last, last] (or [-last, 0] where later keys share bucket 0), so that a
// vector anywhere reads eight places in a row, far ones the end values.  (Four copies, each
// a place further, for two aligned 16-byte reads in the place of eight words: 8 x 12 x 1024 x
// 1024 scores 42.6 us, so 43.3.)
__host__ __device__ __forceinline__ int line_places(int span) { return span + 17; }

__device__ __forceinline__ int clamped(int64_t x, int lo, int hi)
{
    return x < lo ? lo : x > hi ? hi : static_cast<int>(x);
}

// The bucket among one direction's of a distance >= 0.
__device__ __forceinline__ int bucket_of(const Borders& B, int distance)
{
    int lo = 0, hi = B.n; // the last border that is not beyond it
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (B.at[mid] <= distance)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

template <typename T, bool kScores>
__global__ void __launch_bounds__(kThreads)
forward_kernel(const __grid_constant__ Geometry G, const __grid_constant__ Borders B,
               const void* __restrict__ table, int32_t table_type, const T* scores, T* out,
               int lanes_log2, int rows_per_block, int tiles, int same_lead)
{
    extern __shared__ float line[];
    constexpr int kAhead = kScores ? 4 : 1; // vectors of a thread in flight
    const int64_t plane = blockIdx.x / tiles;
    const int h = static_cast<int>(plane % G.heads), b = static_cast<int>(plane / G.heads);
    const int rows = length_of(G.q_lengths, b, G.q_len);
    const int row0 = static_cast<int>(blockIdx.x % tiles) * rows_per_block;
    const int row1 = min(row0 + rows_per_block, rows);
    if (row0 >= row1) return;
    const int keys = length_of(G.k_lengths, b, G.k_len);
    const int64_t start = start_of(G, b);
    const int last = B.at[B.n - 1];
    const int span = B.both ? 2 * last : last;
    const int places = line_places(span);
    // A thread to a place: all loads of the table at once (a warp to a bucket takes one after
    // another: 32 x 2048 x 2048 41.9 us in the place of 40.6).
    for (int k = threadIdx.x; k < places; k += kThreads) {
        const int d = min(max(k - 8, 0), span) - last;
        const int bucket = bucket_of(B, d < 0 ? -d : d) + (d > 0 ? B.n : 0);
        float x[1];
        dev::load_any<1>(table, table_type, static_cast<int64_t>(bucket) * G.heads + h, x);
        line[k] = x[0];
    }
    __syncthreads();

    const int lanes = 1 << lanes_log2;
    const int lane = threadIdx.x & (lanes - 1);
    for (int i = row0 + (threadIdx.x >> lanes_log2); i < row1; i += kThreads >> lanes_log2) {
        T* o = out + plane * G.out_plane + i * G.out_stride;
        const T* s = kScores ? scores + plane * G.in_plane + i * G.in_stride : nullptr;
        const int lead = static_cast<int>((reinterpret_cast<uintptr_t>(o) & 15u) / sizeof(T));
        const int64_t at = start + i; // the query's position
        const int end = G.causal ? clamped(at + 1, 0, keys) : keys; // masked from here on
        const int place = clamped(8 + last - at, -(1 << 29), 1 << 29); // of column 0
        for (int c = lane * 8 - lead; c < G.k_len; c += kAhead * 8 * lanes) {
            Raw8<T> raw[kAhead];
            if (kScores && same_lead) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const int j0 = c + k * 8 * lanes;
                    if (j0 >= 0 && j0 + 8 <= end) dev::stream_raw8(s + j0, raw[k]);
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int j0 = c + k * 8 * lanes;
                if (j0 >= G.k_len) break;
                float x[8];
                if (j0 >= end) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = -INFINITY;
                } else {
                    const float* from = line + min(max(j0 + place, 0), span + 9);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = from[e];
                    if (kScores) {
                        if (same_lead && j0 >= 0 && j0 + 8 <= end) {
                            float y[8];
                            dev::unpack8(raw[k], y);
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] += y[e];
                        } else {
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                if (j0 + e >= 0 && j0 + e < end) x[e] += dev::load1(s + j0 + e);
                        }
                    }
                    if (j0 + 8 > end) {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (j0 + e >= end) x[e] = -INFINITY;
                    }
                }
                if (j0 >= 0 && j0 + 8 <= G.k_len) {
                    dev::store8_stream(o + j0, x);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (j0 + e >= 0 && j0 + e < G.k_len) dev::store1(o + j0 + e, x[e]);
                }
            }
        }
    }
}

// ----------------------------------------------------------------- backward
constexpr int kWarps = 8;
constexpr int kSums = 15;         // diagonals of a slot
constexpr int kBand = 8 * 32 + 7; // diagonals of a warp's 32 slots

// Rows come in groups of eight: group g holds the rows 8g - r .. 8g - r + 7, where
// r = start mod 8, so that row 8g - r + k stands k places into its octet of
// positions.  Row i's vector u lies in slot u - (r + i + lead_i) / 8 (rounded down); its
// element e is on diagonal 8 * (slot - floor(start / 8)) + e - (r + i + lead_i) mod 8.
// A block takes one band of 32 slots, a part of the groups that meet it and a part
// of the batch; partial sums are [heads][parts][buckets].  (4 warps to a block in the place of
// 8: 187 us for 4 x 32 x 2048 x 2048, 40 for 16 x 12 x 333 x 333; 178 and 34.)
struct Split {
    int32_t top, bands; // band k holds the slots top - 32k - 31 .. top - 32k
    int32_t groups, group_parts, groups_per_part;
    int32_t batch_parts, batch_per_part;
    int32_t parts, buckets;
};

template <int kPhase>
__device__ __forceinline__ void add_diagonals(const float (&x)[8], float (&acc)[kSums])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e - kPhase + 7] += x[e];
}

template <typename T>
__device__ __forceinline__ int lead_of(const T* p)
{
    return static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15u) / sizeof(T));
}
// Elements f .. l - 1 of a vector, +0 in the place of the others.
__device__ __forceinline__ uint32_t keep_pair(uint32_t w, int e, int f, int l)
{
    return w & ((e >= f && e < l ? 0xFFFFu : 0u) | (e + 1 >= f && e + 1 < l ? 0xFFFF0000u : 0u));
}
__device__ __forceinline__ void keep_inside(Raw8<Bf16>& r, int f, int l)
{
    r.a = make_uint4(keep_pair(r.a.x, 0, f, l), keep_pair(r.a.y, 2, f, l), keep_pair(r.a.z, 4, f, l),
                     keep_pair(r.a.w, 6, f, l));
}
__device__ __forceinline__ void keep_inside(Raw8<float>& r, int f, int l)
{
    auto keep = [&](float x, int e) { return e >= f && e < l ? x : 0.0f; };
    r.a = make_float4(keep(r.a.x, 0), keep(r.a.y, 1), keep(r.a.z, 2), keep(r.a.w, 3));
    r.b = make_float4(keep(r.b.x, 4), keep(r.b.y, 5), keep(r.b.z, 6), keep(r.b.w, 7));
}
// The elements of a vector at column j0 that lie in columns 0 .. keys - 1, one by one.
__device__ __forceinline__ void load_inside(const Bf16* at, int j0, int keys, Raw8<Bf16>& r)
{
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = j0 + e >= 0 && j0 + e < keys ? at[e].bits : 0u;
        w[e / 2] = e % 2 ? w[e / 2] | b << 16 : b;
    }
    r.a = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void load_inside(const float* at, int j0, int keys, Raw8<float>& r)
{
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = j0 + e >= 0 && j0 + e < keys ? at[e] : 0.0f;
    r.a = make_float4(x[0], x[1], x[2], x[3]);
    r.b = make_float4(x[4], x[5], x[6], x[7]);
}

// kAligned: every row starts at a 16-byte boundary, so that a row's place in its
// group is its phase.
template <typename T, bool kAligned>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 2 ? 3 : 2)
backward_kernel(const __grid_constant__ Geometry G, const __grid_constant__ Borders B,
                const __grid_constant__ Split S, const T* __restrict__ dout,
                const T* __restrict__ dout_end, float* __restrict__ partial)
{
    __shared__ float diag[kWarps][kBand + 1];
    __shared__ float total[kBand + 1];
    __shared__ float sums[kMaxBuckets];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int rest = blockIdx.x;
    const int band = rest % S.bands;
    rest /= S.bands;
    const int group_part = rest % S.group_parts;
    const int b0 = rest / S.group_parts * S.batch_per_part;
    const int b1 = min(b0 + S.batch_per_part, G.batch);
    const int h = blockIdx.y;
    const int low = S.top - 32 * band - 31; // the band's first slot
    const int slot = low + lane;
    for (int q = threadIdx.x; q < S.buckets; q += 32 * kWarps) sums[q] = 0.0f;
    float acc[kSums];
#pragma unroll
    for (int k = 0; k < kSums; ++k) acc[k] = 0.0f;

    // the sums of the diagonals to the sums of their buckets: a thread takes a bucket of a
    // few diagonals, a warp one of many
    auto flush = [&](int64_t octets_before) {
        float* mine = diag[warp];
        if (lane < 7) mine[lane] = 0.0f;
#pragma unroll
        for (int k = 7; k < kSums; ++k) mine[8 * lane + k] = acc[k];
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 7; ++k) mine[8 * lane + k] += acc[k]; // the slot before's
#pragma unroll
        for (int k = 0; k < kSums; ++k) acc[k] = 0.0f;
        __syncthreads();
        const int64_t d0 = 8 * (low - octets_before) - 7; // the diagonal of total[0]
        for (int t = threadIdx.x; t < kBand; t += 32 * kWarps) {
            float x = 0.0f;
            if (!G.causal || d0 + t <= 0) {
#pragma unroll
                for (int w = 0; w < kWarps; ++w) x += diag[w][t];
            }
            total[t] = x;
        }
        __syncthreads();
        constexpr int64_t kFar = int64_t(1) << 60;
        auto interval = [&](int q, int& t0, int& t1) {
            int64_t from, to; // the bucket's diagonals
            if (q < B.n) {
                from = q + 1 < B.n ? 1 - static_cast<int64_t>(B.at[q + 1]) : -kFar;
                to = q == 0 && !B.both ? kFar : 1 - static_cast<int64_t>(B.at[q]);
            } else {
                from = B.at[q - B.n] > 1 ? B.at[q - B.n] : 1;
                to = q - B.n + 1 < B.n ? B.at[q - B.n + 1] : kFar;
            }
            t0 = clamped(from - d0, 0, kBand);
            t1 = clamped(to - d0, 0, kBand);
        };
        // buckets q0 .. q0 + 31 are this warp's, lane by lane
        for (int q0 = 32 * warp; q0 < S.buckets; q0 += 32 * kWarps) {
            int t0 = 0, t1 = 0;
            if (q0 + lane < S.buckets) interval(q0 + lane, t0, t1);
            if (t1 - t0 <= 16) {
                float x = 0.0f;
                for (int t = t0; t < t1; ++t) x += total[t];
                if (t0 < t1) sums[q0 + lane] += x;
            }
            unsigned many = __ballot_sync(0xFFFFFFFFu, t1 - t0 > 16);
            while (many) {
                const int l = __ffs(many) - 1;
                many &= many - 1;
                const int from = __shfl_sync(0xFFFFFFFFu, t0, l), to = __shfl_sync(0xFFFFFFFFu, t1, l);
                float x = 0.0f;
                for (int t = from + lane; t < to; t += 32) x += total[t];
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, off);
                if (lane == 0) sums[q0 + l] += x;
            }
        }
    };

    for (int b = b0; b < b1; ++b) {
        const int64_t start = start_of(G, b);
        const int r = static_cast<int>(start & 7);
        const int64_t octets_before = start >> 3;
        const int rows = length_of(G.q_lengths, b, G.q_len);
        const int keys = length_of(G.k_lengths, b, G.k_len);
        const T* plane = dout + (static_cast<int64_t>(b) * G.heads + h) * G.in_plane;
        // later keys' slots are not read under a causal mask (of slot 0 the later diagonals
        // are left out at the end)
        const bool counted = !G.causal || slot <= octets_before;
        // groups with vectors in this band
        const int most = (keys + 14) / 8; // vectors of a row, at most
        int g0 = max(0, -low - 32), g1 = min(S.groups, most - low);
        g0 += group_part * S.groups_per_part;
        g1 = min(g1, g0 + S.groups_per_part);
        for (int g = g0 + warp; g < g1; g += kWarps) {
            const int i0 = 8 * g - r;
            const T* first = plane + i0 * G.in_stride; // row i0, where there is one
            Raw8<T> raw[8];
            int place[8]; // of a row: its lead and its place in the group, phase and carry
            // All eight rows' vectors whole in all lanes: no checks.  A row's lead may
            // move its vectors by one.
            const int u0 = low + g, u1 = u0 + 31 + (kAligned ? 0 : 1);
            const bool inner = i0 >= 0 && i0 + 8 <= rows && u0 >= (kAligned ? 0 : 1) &&
                               8 * u1 + 8 <= keys && (!G.causal || low + 31 <= octets_before);
            if (inner) {
                const T* at = first + 8 * (slot + g);
#pragma unroll
                for (int k = 0; k < 8; ++k, at += G.in_stride) {
                    const int lead = kAligned ? 0 : lead_of(at);
                    place[k] = k + lead;
                    dev::stream_raw8(kAligned ? at : at - lead + (place[k] & 8), raw[k]);
                }
            } else {
                unsigned edge = 0; // bit k: not all of vector k counts
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const T* row = first + k * G.in_stride;
                    const int lead = kAligned ? 0 : lead_of(row);
                    place[k] = k + lead;
                    const int u = slot + g + (place[k] >> 3);
                    const int j0 = 8 * u - lead;
                    raw[k] = Raw8<T>{};
                    if (counted && i0 + k >= 0 && i0 + k < rows && u >= 0 && j0 < keys) {
                        if (j0 < 0 || j0 + 8 > keys) edge |= 1u << k;
                        const T* at = row + j0;
                        if (at >= dout && at + 8 <= dout_end)
                            dev::stream_raw8(at, raw[k]);
                        else // not all of it is the tensor's
                            load_inside(at, j0, keys, raw[k]);
                    }
                }
                if (__any_sync(0xFFFFFFFFu, edge)) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        if (edge & (1u << k)) {
                            const int j0 = 8 * (slot + g + (place[k] >> 3)) - (place[k] - k);
                            keep_inside(raw[k], -j0, keys - j0);
                        }
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                float x[8];
                dev::unpack8(raw[k], x);
                switch (kAligned ? k : place[k] & 7) { // the same in all lanes
                case 0: add_diagonals<0>(x, acc); break;
                case 1: add_diagonals<1>(x, acc); break;
                case 2: add_diagonals<2>(x, acc); break;
                case 3: add_diagonals<3>(x, acc); break;
                case 4: add_diagonals<4>(x, acc); break;
                case 5: add_diagonals<5>(x, acc); break;
                case 6: add_diagonals<6>(x, acc); break;
                default: add_diagonals<7>(x, acc);
                }
            }
        }
        if (G.starts || b + 1 == b1) flush(octets_before);
    }
    __syncthreads();
    float* to = partial + (static_cast<int64_t>(h) * S.parts + blockIdx.x) * S.buckets;
    for (int q = threadIdx.x; q < S.buckets; q += 32 * kWarps) to[q] = sums[q];
}

// One block adds the parts of 32 buckets of one head.
__global__ void __launch_bounds__(32 * kWarps)
reduce_kernel(const float* __restrict__ partial, int parts, int buckets, int heads, void* dtable,
              int32_t type, int accumulate)
{
    __shared__ float sums[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int q = blockIdx.x * 32 + lane, h = blockIdx.y;
    // launched while the blocks of the kernel before drain
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float x = 0.0f;
    if (q < buckets) {
        const float* from = partial + static_cast<int64_t>(h) * parts * buckets + q;
#pragma unroll 4
        for (int p = warp; p < parts; p += kWarps) x += from[static_cast<int64_t>(p) * buckets];
    }
    sums[warp][lane] = x;
    __syncthreads();
    if (warp == 0 && q < buckets) {
        float all[1] = {0.0f};
#pragma unroll
        for (int w = 0; w < kWarps; ++w) all[0] += sums[w][lane];
        const int64_t at = static_cast<int64_t>(q) * heads + h;
        if (accumulate) {
            float old[1];
            dev::load_any<1>(dtable, type, at, old);
            all[0] += old[0];
        }
        dev::store_any<1>(dtable, type, at, all);
    }
}

// --------------------------------------------------------------------- host
// A number as digits to the base 2^32, for the comparison of powers: at most 256
// factors below 2^14 and as many below 2^9.
struct Digits {
    uint32_t d[256] = {1};
    int n = 1;
    Digits& times(int64_t f, int exponent)
    {
        for (int k = 0; k < exponent; ++k) {
            uint64_t carry = 0;
            for (int i = 0; i < n; ++i) {
                carry += d[i] * static_cast<uint64_t>(f);
                d[i] = static_cast<uint32_t>(carry);
                carry >>= 32;
            }
            if (carry && n < 256) d[n++] = static_cast<uint32_t>(carry);
        }
        return *this;
    }
    bool operator>=(const Digits& o) const
    {
        if (n != o.n) return n > o.n;
        for (int i = n - 1; i >= 0; --i)
            if (d[i] != o.d[i]) return d[i] > o.d[i];
        return true;
    }
};

// Part j of the logarithmic ones begins at the smallest n with
// (n / half)^parts >= (distance / half)^j: at the next whole number of the power's
// double, unless that is so near a whole number that only whole numbers tell.
Borders make_borders(int32_t buckets, int32_t both, int64_t distance)
{
    Borders B = {};
    B.n = both ? buckets / 2 : buckets;
    B.both = both;
    const int half = B.n / 2, parts = B.n - half;
    for (int i = 0; i < half; ++i) B.at[i] = static_cast<int16_t>(i);
    const double step = std::log(static_cast<double>(distance) / half) / parts;
    for (int j = 0; j < parts; ++j) {
        const double x = half * std::exp(j * step);
        int64_t n = static_cast<int64_t>(std::floor(x + 0.5));
        if (std::fabs(x - static_cast<double>(n)) > 1e-6)
            n = static_cast<int64_t>(std::ceil(x));
        else if (!(Digits().times(n, parts).times(half, j) >=
                   Digits().times(distance, j).times(half, parts)))
            ++n;
        B.at[half + j] = static_cast<int16_t>(n);
    }
    return B;
}

bool sizes_ok(int64_t batch, int64_t heads, int64_t q_len, int64_t k_len, int32_t buckets)
{
    return batch >= 0 && heads >= 1 && heads <= 65535 && q_len >= 0 && q_len <= kMaxLen &&
           k_len >= 0 && k_len <= kMaxLen && batch <= (int64_t(1) << 30) &&
           batch * heads <= (int64_t(1) << 30) && buckets >= 2 && buckets <= kMaxBuckets;
}

int check_relpos(const zero_relpos_t* r, const int32_t* starts, const int32_t* q_lengths,
                 const int32_t* k_lengths)
{
    if (!r || !sizes_ok(r->batch, r->heads, r->q_len, r->k_len, r->buckets) ||
        !float_type(r->table_type) || !float_type(r->type) ||
        (r->bidirectional != 0 && r->bidirectional != 1) || (r->causal != 0 && r->causal != 1))
        return ZERO_EINVAL;
    if (r->bidirectional && (r->buckets % 2 != 0 || r->buckets < 4)) return ZERO_EINVAL;
    const int32_t half = (r->bidirectional ? r->buckets / 2 : r->buckets) / 2;
    if (r->max_distance <= half || r->max_distance > kMaxDistance) return ZERO_EINVAL;
    if (r->start > kMaxStart || r->start < -kMaxStart) return ZERO_EINVAL;
    if (!aligned_to(starts, 4) || !aligned_to(q_lengths, 4) || !aligned_to(k_lengths, 4))
        return ZERO_EALIGN;
    return ZERO_OK;
}

Geometry geometry(const zero_relpos_t* r, const int32_t* starts, const int32_t* q_lengths,
                  const int32_t* k_lengths)
{
    Geometry G = {};
    G.start = r->start;
    G.starts = starts;
    G.q_lengths = q_lengths;
    G.k_lengths = k_lengths;
    G.batch = static_cast<int32_t>(r->batch);
    G.heads = static_cast<int32_t>(r->heads);
    G.q_len = static_cast<int32_t>(r->q_len);
    G.k_len = static_cast<int32_t>(r->k_len);
    G.causal = r->causal;
    return G;
}

template <typename T>
int launch_forward(const Geometry& G, const Borders& B, const void* table, int32_t table_type,
                   const void* scores, void* out, cudaStream_t stream)
{
    constexpr int kUnit = 16 / sizeof(T);
    const int vecs = (G.k_len + kUnit - 1 + 7) / 8;
    int log2 = 0;
    while (log2 < 5 && (1 << log2) < vecs) ++log2;
    // blocks of at least 64 K places, and 16 for each of the line, which is laid out in each
    // (512 buckets up to 8192, 32 x 2048 x 2048: 185 us, 265 without the latter)
    const int last = B.at[B.n - 1];
    const int span = B.both ? 2 * last : last;
    const int per_pass = kThreads >> log2;
    const int64_t least = std::max<int64_t>(65536, 16 * line_places(span));
    int64_t rows = (least + G.k_len - 1) / G.k_len;
    rows = (rows + per_pass - 1) / per_pass * per_pass;
    if (rows > G.q_len) rows = G.q_len;
    const int64_t tiles = (G.q_len + rows - 1) / rows;
    const int64_t blocks = tiles * G.batch * G.heads;
    if (blocks > 0x7FFFFFFF) return ZERO_EINVAL;
    const int same = scores && ((reinterpret_cast<uintptr_t>(scores) ^ reinterpret_cast<uintptr_t>(out)) & 15u) == 0 &&
                     (G.in_stride - G.out_stride) % kUnit == 0 &&
                     (G.in_plane - G.out_plane) % kUnit == 0;
    const size_t bytes = 4 * static_cast<size_t>(line_places(span));
    auto start = [&](auto kernel) {
        // the limit that every block has without asking is 48 KB
        if (bytes > 48 * 1024 && !allow_shared(reinterpret_cast<const void*>(kernel),
                                               4 * static_cast<size_t>(line_places(2 * kMaxDistance))))
            return ZERO_ECUDA;
        kernel<<<static_cast<unsigned>(blocks), kThreads, bytes, stream>>>(
            G, B, table, table_type, static_cast<const T*>(scores), static_cast<T*>(out), log2,
            static_cast<int>(rows), static_cast<int>(tiles), same);
        return cuda_status(cudaGetLastError());
    };
    return scores ? start(forward_kernel<T, true>) : start(forward_kernel<T, false>);
}

constexpr int64_t kResident = 152 * 3; // blocks at once

// The split of a call's work: by its sizes alone (with a causal mask also by start).
Split split(int64_t batch, int64_t heads, int64_t q_len, int64_t k_len, int32_t buckets,
            bool below, int64_t octets_before)
{
    Split S = {};
    S.buckets = buckets;
    if (batch == 0 || q_len == 0 || k_len == 0) return S;
    const int64_t vectors = (k_len + 14) / 8;       // of a row, with the row's lead of up to 7
    const int64_t bottom = -((7 + q_len - 1 + 7) / 8);
    int64_t top = vectors - 1;
    if (below && octets_before < top) top = octets_before;
    if (top < bottom) return S;
    S.top = static_cast<int32_t>(top);
    S.bands = static_cast<int32_t>((top - bottom + 32) / 32);
    S.groups = static_cast<int32_t>((q_len + 7 + 7) / 8);
    // groups that meet one band
    const int64_t meet = std::min<int64_t>(S.groups, vectors + 32);
    const int64_t planes = heads * S.bands * batch;
    // at least two rounds of blocks where that leaves a warp four groups, and 16 at most
    int64_t parts = (2 * kResident + planes - 1) / planes;
    parts = std::max<int64_t>(1, std::min<int64_t>(parts, meet / (4 * kWarps)));
    S.groups_per_part = static_cast<int32_t>((meet + parts - 1) / parts);
    S.group_parts = static_cast<int32_t>((meet + S.groups_per_part - 1) / S.groups_per_part);
    const int64_t per = std::min<int64_t>(batch, std::max<int64_t>(1, planes / (8 * kResident)));
    S.batch_per_part = static_cast<int32_t>(per);
    S.batch_parts = static_cast<int32_t>((batch + per - 1) / per);
    S.parts = S.bands * S.group_parts * S.batch_parts;
    return S;
}

// The most parts of a head that split() gives for these sizes.  With p = heads * bands *
// batch below 2 * kResident they are bands * batch * ceil(2 * kResident / p) at most, less
// than 4 * kResident / heads; up to 16 * kResident they are bands * batch; beyond, bands *
// ceil(batch / floor(p / (8 * kResident))), less than 16 * kResident / heads + bands.  A
// causal mask leaves fewer bands.
int64_t most_parts(int64_t batch, int64_t heads, int64_t q_len, int64_t k_len, int32_t buckets)
{
    return (16 * kResident + heads - 1) / heads +
           split(batch, heads, q_len, k_len, buckets, false, 0).bands + 1;
}

template <typename T>
int launch_backward(const Geometry& G, const Borders& B, const Split& S, const void* dout,
                    float* partial, cudaStream_t stream)
{
    const auto* from = static_cast<const T*>(dout);
    const T* end = from + (static_cast<int64_t>(G.batch) * G.heads - 1) * G.in_plane +
                   (G.q_len - 1) * G.in_stride + G.k_len;
    constexpr int kUnit = 16 / sizeof(T);
    const dim3 grid(static_cast<unsigned>(S.parts), static_cast<unsigned>(G.heads));
    // 4 x 32 x 2048 x 2048 bf16: 179 us, by the code for any row 210; fp32 (half the batch) takes
    // 174 by that and would take 178
    if (sizeof(T) == 2 && aligned16(dout) && G.in_stride % kUnit == 0 && G.in_plane % kUnit == 0)
        backward_kernel<Bf16, true><<<grid, 32 * kWarps, 0, stream>>>(
            G, B, S, reinterpret_cast<const Bf16*>(from), reinterpret_cast<const Bf16*>(end), partial);
    else
        backward_kernel<T, false><<<grid, 32 * kWarps, 0, stream>>>(G, B, S, from, end, partial);
    return cuda_status(cudaGetLastError());
}

} // namespace
} // namespace zero

using namespace zero;

extern "C" int zero_relpos_forward(const zero_relpos_t* relpos, const void* table,
                                   const int32_t* starts, const int32_t* q_lengths,
                                   const int32_t* k_lengths, const void* scores,
                                   int64_t scores_stride, void* out, int64_t out_stride,
                                   cudaStream_t stream)
{
    const int rc = check_relpos(relpos, starts, q_lengths, k_lengths);
    if (rc != ZERO_OK) return rc;
    if (relpos->batch == 0 || relpos->q_len == 0 || relpos->k_len == 0) return ZERO_OK;
    if (!table || !out || out_stride < relpos->k_len || out_stride > kMaxStride ||
        (scores && (scores_stride < relpos->k_len || scores_stride > kMaxStride)) ||
        (scores == out && scores_stride != out_stride))
        return ZERO_EINVAL;
    const int tb = type_bytes(relpos->type);
    if (!aligned_to(table, type_bytes(relpos->table_type)) || !aligned_to(scores, tb) ||
        !aligned_to(out, tb))
        return ZERO_EALIGN;
    Geometry G = geometry(relpos, starts, q_lengths, k_lengths);
    G.out_stride = out_stride;
    G.in_stride = scores_stride;
    G.out_plane = out_stride * relpos->q_len;
    G.in_plane = scores_stride * relpos->q_len;
    const Borders B = make_borders(relpos->buckets, relpos->bidirectional, relpos->max_distance);
    return relpos->type == ZERO_TYPE_BF16
               ? launch_forward<Bf16>(G, B, table, relpos->table_type, scores, out, stream)
               : launch_forward<float>(G, B, table, relpos->table_type, scores, out, stream);
}

extern "C" int64_t zero_relpos_scratch_bytes(int64_t batch, int64_t heads, int64_t q_len,
                                             int64_t k_len, int32_t buckets)
{
    if (!sizes_ok(batch, heads, q_len, k_len, buckets)) return ZERO_EINVAL;
    return (heads * most_parts(batch, heads, q_len, k_len, buckets) * buckets * 4 + 15) / 16 * 16;
}

extern "C" int zero_relpos_backward(const zero_relpos_t* relpos, const int32_t* starts,
                                    const int32_t* q_lengths, const int32_t* k_lengths,
                                    const void* dout, int64_t dout_stride, void* dtable,
                                    int32_t accumulate, void* scratch, int64_t scratch_bytes,
                                    cudaStream_t stream)
{
    int rc = check_relpos(relpos, starts, q_lengths, k_lengths);
    if (rc != ZERO_OK) return rc;
    if (!dtable || !scratch || (accumulate != 0 && accumulate != 1)) return ZERO_EINVAL;
    const bool empty = relpos->batch == 0 || relpos->q_len == 0 || relpos->k_len == 0;
    if (!empty && (!dout || dout_stride < relpos->k_len || dout_stride > kMaxStride))
        return ZERO_EINVAL;
    const int64_t need = zero_relpos_scratch_bytes(relpos->batch, relpos->heads, relpos->q_len,
                                                   relpos->k_len, relpos->buckets);
    if (need < 0 || scratch_bytes < need) return ZERO_EINVAL;
    if (!aligned_to(dout, type_bytes(relpos->type)) ||
        !aligned_to(dtable, type_bytes(relpos->table_type)) || !aligned16(scratch))
        return ZERO_EALIGN;
    Geometry G = geometry(relpos, starts, q_lengths, k_lengths);
    G.in_stride = dout_stride;
    G.in_plane = dout_stride * relpos->q_len;
    const Borders B = make_borders(relpos->buckets, relpos->bidirectional, relpos->max_distance);
    const Split S = split(relpos->batch, relpos->heads, relpos->q_len, relpos->k_len,
                          relpos->buckets, relpos->causal && !starts, relpos->start >> 3);
    if (S.parts > most_parts(relpos->batch, relpos->heads, relpos->q_len, relpos->k_len,
                             relpos->buckets))
        return ZERO_EINVAL;
    auto* partial = static_cast<float*>(scratch);
    if (S.parts > 0) {
        rc = relpos->type == ZERO_TYPE_BF16
                 ? launch_backward<Bf16>(G, B, S, dout, partial, stream)
                 : launch_backward<float>(G, B, S, dout, partial, stream);
        if (rc != ZERO_OK) return rc;
    } else if (accumulate) {
        return ZERO_OK;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((relpos->buckets + 31) / 32),
                       static_cast<unsigned>(relpos->heads));
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = S.parts > 0 ? 1 : 0;
    return cuda_status(cudaLaunchKernelEx(&cfg, reduce_kernel, partial, S.parts, relpos->buckets,
                                          static_cast<int>(relpos->heads), dtable,
                                          relpos->table_type, accumulate));
}
