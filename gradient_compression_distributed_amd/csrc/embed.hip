// embed.hip -- embedding lookup with scaling, and its gradient by sorted
// tokens, for gfx950.
//
//   lookup   out[i] = round(scale * E[tok_i])          (one rounding)
//   gradient dE[v]  = scale * sum over i with tok_i = v of g[i]
//
// A token outside [0, V) is padding: a zero row, no gradient.
//
// The gradient is a sum over positions that share a token.  Atomics would
// add in an order that changes from call to call; here the positions are
// sorted by token first (a stable radix sort, so equal tokens keep their
// order), and every sum runs over sorted positions in a fixed order.
#include <algorithm>

#include "gcq_device.h"
#include "gcq_lm.h"

namespace gcq {

namespace {

using namespace lm;

// ------------------------------------------------------------------ lookup
// L lanes share a row (a power of two up to 256), so a workgroup of 256
// threads copies 256 / L rows at once, R times over, and of each at most
// kLookupTrips vectors a lane: `cols` workgroups share a longer row (16000 rows
// of 8192 float32 131 us, by one workgroup each 145; with one vector a lane
// 136).  The R tokens are loaded together and then the R rows' vectors, so a
// row waits for one load, not for two in turn (32768 rows of 4096 bf16, us for
// R = 1 / 2 / 4 / 8: 80 / 75 / 82 / 83).  Bound by memory: there 268 MB go out
// and 168 MB come in, 97 MB of different rows and 71 MB of frequent ones that
// several XCDs fetch, 5.8 TB/s.  A few rows take a launch (3 us).
template <typename T, typename O>
constexpr int kLookup = kVec<T> < kVec<O> ? kVec<T> : kVec<O>;   // 16 bytes at most on either side
constexpr uint32_t kLookupTrips = 2;

template <typename T, typename O, typename I, int R>
__global__ __launch_bounds__(256) void embed_lookup_kernel(const T *__restrict__ table,
                                                           uint64_t vocab, uint64_t dim,
                                                           uint64_t ld,
                                                           const I *__restrict__ tokens,
                                                           uint64_t n, float scale,
                                                           O *__restrict__ out, uint64_t out_ld,
                                                           uint32_t lanes, uint32_t cols)
{
    constexpr int N = kLookup<T, O>;
    const uint32_t lane = threadIdx.x & (lanes - 1), slots = 256u / lanes;
    const uint64_t block = block_number();
    const uint64_t row0 = block / cols * slots * R + threadIdx.x / lanes;   // then every slots-th
    uint64_t tok[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const uint64_t row = row0 + (uint64_t)r * slots;
        tok[r] = row < n ? (uint64_t)(int64_t)((const GCQ_G I *)tokens)[row] : ~0ull;
    }
    const uint64_t width = (uint64_t)lanes * N * kLookupTrips, c0 = block % cols * width;
    const uint64_t c1 = c0 + width < dim ? c0 + width : dim;
    for (uint64_t c = c0 + (uint64_t)lane * N; c < c1; c += (uint64_t)lanes * N) {
        const int64_t left = (int64_t)(dim - c);
        vec<T, N> v[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            v[r] = (T)0.0f;
            if (tok[r] < vocab)   // a negative token is past any vocab
                v[r] = load_vec<T, N>(table + tok[r] * ld + c, left);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const uint64_t row = row0 + (uint64_t)r * slots;
            fvec<N> f = 0.0f;
            if (tok[r] < vocab)
                f = to_f32<T, N>(v[r]) * scale;   // a padding row stays +0
            if (row < n)
                store_vec<O, N, true>(out + row * out_ld + c, from_f32<O, N>(f), left);
        }
    }
}

// -------------------------------------------------------------------- sort
__device__ __forceinline__ uint32_t key_of(int64_t token, uint64_t vocab)
{
    const uint64_t t = (uint64_t)token;
    return (uint32_t)(t < vocab ? t : vocab);   // padding sorts behind every token
}

// Few positions: each finds its place by counting.  The place of position i
// is the number of positions before it with a key <= its own and of positions
// behind it with a smaller key.  A workgroup holds every key in LDS; Ti lanes
// take a position each, 1024 / Ti groups of lanes a share of the others.
// n^2 comparisons (2 instructions each) cost less than the passes of a radix
// sort, each of them bound by launch and latency, up to kCountSort positions:
// 7 us at 4000; with the rest of a row-sparse gradient of 64 columns 31 us
// against 40 at 6000 and 34 against 40 at 8000, but 38 us against 26 for the
// sort alone at 16384.
constexpr uint32_t kCountSort = 8192;
template <typename I, uint32_t Ti>
__global__ __launch_bounds__(1024) void embed_count_sort_kernel(const I *__restrict__ tokens,
                                                                uint32_t n, uint32_t share,
                                                                uint64_t vocab,
                                                                uint32_t *__restrict__ keys,
                                                                uint32_t *__restrict__ order)
{
    // share * 1024 / Ti keys, those past n never counted
    extern __shared__ __align__(16) uint32_t key_s[];
    __shared__ uint32_t place[Ti];
    const uint32_t tid = threadIdx.x, all = share * (1024u / Ti);
    for (uint32_t j = tid; j < all; j += 1024u)
        key_s[j] = j < n ? key_of(((const GCQ_G I *)tokens)[j], vocab) : 0xFFFFFFFFu;
    if (tid < Ti)
        place[tid] = 0;
    __syncthreads();
    const uint32_t i0 = blockIdx.x * Ti, i = i0 + tid % Ti;
    const uint32_t j0 = tid / Ti * share;
    const uint32_t key = i < n ? key_s[i] : 0u;
    uint32_t count = 0;
    if (j0 + share <= i0 || j0 >= i0 + Ti) {
        const uint32_t below = key + (j0 < i0);   // ahead: <= key; behind: < key
#pragma unroll 4
        for (uint32_t j = 0; j < share; j += 4) {
            const uint4 k = *(const uint4 *)(key_s + j0 + j);
            count += (uint32_t)(k.x < below) + (uint32_t)(k.y < below) + (uint32_t)(k.z < below) +
                     (uint32_t)(k.w < below);
        }
    } else {
        for (uint32_t j = j0; j < j0 + share; ++j)
            count += key_s[j] < key + (j < i);
    }
    if (i < n)
        atomicAdd(&place[tid % Ti], count);   // whole numbers: any order
    __syncthreads();
    if (tid < Ti && i < n && place[tid] < n) {
        keys[place[tid]] = key;
        order[place[tid]] = i;
    }
}

// More: least-significant-digit radix sort of (key, position), digits of at
// most 9 bits, tiles of 2048 positions, two launches a pass.  A wavefront
// ranks 64 keys at a time: a ballot per digit bit gives each lane the lanes
// that share its digit, so the rank is a count of lower lanes plus the
// wavefront's count so far, and equal digits keep their order.  65536 tokens
// of 18 bits: 24 us in four launches of 5 to 7, each a few dependent trips to
// memory that another launch wrote.
constexpr uint32_t kDigitBits = 9, kBins = 1u << kDigitBits;
constexpr uint32_t kSortThreads = 512, kSortItems = 4;
constexpr uint32_t kSortTile = kSortThreads * kSortItems;
// Up to this many tiles each scatter sums the tiles' counts itself; beyond, a
// launch of its own scans them (a scatter's own reading grows with the square).
// Counting every key in each scatter, to save the launch that counts, took
// longer from 10000 positions on: the frequent tokens' LDS atomics collide.
constexpr uint32_t kSumTiles = 128;

__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Ranks this wavefront's Items digits among its earlier ones of equal value;
// cnt[bin] (zero on entry) ends as the wavefront's histogram.  Items with
// digit >= kBins take no part.
template <int Items>
__device__ __forceinline__ void wave_rank(const uint32_t (&digit)[Items], uint32_t bits,
                                          uint32_t *cnt, uint32_t (&rank)[Items])
{
    const uint32_t lane = threadIdx.x & (kWave - 1);
    const uint64_t below = (1ull << lane) - 1u;
    uint64_t peers[Items];
#pragma unroll
    for (int j = 0; j < Items; ++j)
        peers[j] = __ballot(digit[j] < kBins);
    for (uint32_t b = 0; b < bits; ++b) {
#pragma unroll
        for (int j = 0; j < Items; ++j) {
            const bool one = (digit[j] >> b) & 1u;
            const uint64_t m = __ballot(one);
            peers[j] &= one ? m : ~m;
        }
    }
#pragma unroll
    for (int j = 0; j < Items; ++j) {
        const bool in = digit[j] < kBins;
        uint32_t first = 0;
        if (in)
            first = cnt[digit[j]];
        wave_order();   // every lane has read before the count moves
        if (in && (peers[j] & below) == 0)
            cnt[digit[j]] = first + (uint32_t)__popcll(peers[j]);
        wave_order();
        rank[j] = first + (uint32_t)__popcll(peers[j] & below);
    }
}

__device__ __forceinline__ uint32_t wave_scan(uint32_t x)
{
    const uint32_t lane = threadIdx.x & (kWave - 1);
#pragma unroll
    for (int o = 1; o < kWave; o <<= 1) {
        const uint32_t y = __shfl_up(x, o, kWave);
        x += lane >= (uint32_t)o ? y : 0u;
    }
    return x;
}

// Exclusive scan of x over the workgroup's threads; sums: one per wavefront.
template <uint32_t Threads>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *sums, uint32_t &total)
{
    constexpr uint32_t waves = Threads / kWave;
    const uint32_t wave = threadIdx.x / kWave;
    const uint32_t incl = wave_scan(x);
    if ((threadIdx.x & (kWave - 1)) == kWave - 1)
        sums[wave] = incl;
    __syncthreads();
    uint32_t before = 0, all = 0;
#pragma unroll
    for (uint32_t w = 0; w < waves; ++w) {
        before += w < wave ? sums[w] : 0u;
        all += sums[w];
    }
    __syncthreads();
    total = all;
    return before + incl - x;
}

// The tile's digit counts: hist[tile][digit].  First: keys come from the
// tokens.
template <typename I, bool First>
__global__ __launch_bounds__(kSortThreads) void embed_hist_kernel(
    const I *__restrict__ tokens, const uint32_t *__restrict__ keys, uint32_t n, uint64_t vocab,
    uint32_t shift, uint32_t digit_bits, uint32_t *__restrict__ hist)
{
    __shared__ uint32_t cnt[kBins];
    static_assert(kBins == kSortThreads, "a thread per digit");
    const uint32_t mask = (1u << digit_bits) - 1u, tid = threadIdx.x;
    const uint64_t t0 = (uint64_t)blockIdx.x * kSortTile;
    uint32_t k[kSortItems];
#pragma unroll
    for (uint32_t j = 0; j < kSortItems; ++j) {
        const uint64_t i = t0 + tid + kSortThreads * j;
        k[j] = i >= n ? 0u : First ? key_of(((const GCQ_G I *)tokens)[i], vocab) : keys[i];
    }
    cnt[tid] = 0;
    __syncthreads();
#pragma unroll
    for (uint32_t j = 0; j < kSortItems; ++j)
        if (t0 + tid + kSortThreads * j < n)
            atomicAdd(&cnt[(k[j] >> shift) & mask], 1u);   // whole numbers: any order
    __syncthreads();
    hist[(uint64_t)blockIdx.x * kBins + tid] = cnt[tid];
}

// In place per digit: each tile's count becomes the count in earlier tiles,
// the row behind the tiles the digit's total.  64 digits per workgroup, 16
// threads a digit over consecutive shares of the tiles.
__global__ __launch_bounds__(1024) void embed_hist_scan_kernel(uint32_t *__restrict__ hist,
                                                               uint32_t tiles)
{
    __shared__ uint32_t share[16][kWave];
    const uint32_t lane = threadIdx.x & (kWave - 1), part = threadIdx.x / kWave;
    uint32_t *h = hist + blockIdx.x * kWave + lane;
    const uint32_t each = (tiles + 15u) / 16u;
    const uint32_t t0 = part * each < tiles ? part * each : tiles;
    const uint32_t t1 = t0 + each < tiles ? t0 + each : tiles;
    uint32_t sum = 0;
#pragma unroll 8
    for (uint32_t t = t0; t < t1; ++t)
        sum += h[(uint64_t)t * kBins];
    share[part][lane] = sum;
    __syncthreads();
    uint32_t x = 0, all = 0;
    for (uint32_t p = 0; p < 16; ++p) {
        x += p < part ? share[p][lane] : 0u;
        all += share[p][lane];
    }
    for (uint32_t t = t0; t < t1; ++t) {
        const uint32_t v = h[(uint64_t)t * kBins];
        h[(uint64_t)t * kBins] = x;
        x += v;
    }
    if (part == 0)
        h[(uint64_t)tiles * kBins] = all;
}

// Scanned: the counts went through embed_hist_scan_kernel.
template <typename I, bool First, bool Scanned>
__global__ __launch_bounds__(kSortThreads) void embed_scatter_kernel(
    const I *__restrict__ tokens, const uint32_t *__restrict__ keys_in,
    const uint32_t *__restrict__ order_in, uint32_t n, uint64_t vocab, uint32_t shift,
    uint32_t digit_bits, const uint32_t *__restrict__ hist, uint32_t tiles,
    uint32_t *__restrict__ keys_out, uint32_t *__restrict__ order_out)
{
    constexpr uint32_t waves = kSortThreads / kWave;
    __shared__ uint32_t cnt[waves][kBins], sums[waves];
    const uint32_t mask = (1u << digit_bits) - 1u, tid = threadIdx.x;
    const uint32_t lane = tid & (kWave - 1), wave = tid / kWave;
    const uint64_t at = (uint64_t)blockIdx.x * kSortTile + wave * kWave * kSortItems + lane;
    uint32_t key[kSortItems], pos[kSortItems], rank[kSortItems], digit[kSortItems];
#pragma unroll
    for (uint32_t j = 0; j < kSortItems; ++j) {
        const uint64_t i = at + kWave * j;
        key[j] = 0;
        pos[j] = (uint32_t)i;
        if (i < n) {
            key[j] = First ? key_of(((const GCQ_G I *)tokens)[i], vocab) : keys_in[i];
            if (!First)
                pos[j] = order_in[i];
        }
    }
    // digit tid: its count in all tiles, and in earlier ones
    uint32_t before = 0, all = 0;
    if constexpr (Scanned) {
        before = hist[(uint64_t)blockIdx.x * kBins + tid];
        all = hist[(uint64_t)tiles * kBins + tid];
    } else {
#pragma unroll 16
        for (uint32_t t = 0; t < tiles; ++t) {
            const uint32_t c = hist[(uint64_t)t * kBins + tid];
            before += t < blockIdx.x ? c : 0u;
            all += c;
        }
    }
#pragma unroll
    for (uint32_t w = 0; w < waves; ++w)
        cnt[w][tid] = 0;
    uint32_t total;
    before += block_scan<kSortThreads>(all, sums, total);   // and a barrier
#pragma unroll
    for (uint32_t j = 0; j < kSortItems; ++j)
        digit[j] = at + kWave * j < n ? (key[j] >> shift) & mask : kBins;
    wave_rank<kSortItems>(digit, digit_bits, cnt[wave], rank);
    __syncthreads();
    uint32_t c[waves];
#pragma unroll
    for (uint32_t w = 0; w < waves; ++w)
        c[w] = cnt[w][tid];
#pragma unroll
    for (uint32_t w = 0; w < waves; ++w) {
        cnt[w][tid] = before;
        before += c[w];
    }
    __syncthreads();
#pragma unroll
    for (uint32_t j = 0; j < kSortItems; ++j) {
        if (digit[j] < kBins) {
            const uint32_t to = cnt[wave][digit[j]] + rank[j];
            if (to < n) {
                keys_out[to] = key[j];
                order_out[to] = pos[j];
            }
        }
    }
}

// ---------------------------------------------------------------- gradient
// Up to here one workgroup counts the segment starts (8 positions a thread,
// the shortest run), beyond it a launch per tile and a scan.
constexpr uint32_t kSmallStarts = 8192;
// Segment starts before each run of sorted positions (within its tile), and
// each tile's count.
__global__ __launch_bounds__(256) void embed_starts_kernel(const uint32_t *__restrict__ keys,
                                                           uint32_t n, uint32_t vocab, uint32_t run,
                                                           uint32_t *__restrict__ starts,
                                                           uint32_t *__restrict__ tiles)
{
    __shared__ uint32_t sums[256 / kWave];
    constexpr uint32_t per = kEmbedTile / 256u;
    const uint64_t i0 = (uint64_t)blockIdx.x * kEmbedTile + threadIdx.x * per;
    uint32_t mine = 0;
    uint32_t last = i0 && i0 < n ? keys[i0 - 1] : 0xFFFFFFFFu;
#pragma unroll
    for (uint32_t j = 0; j < per; ++j) {
        if (i0 + j < n) {
            const uint32_t k = keys[i0 + j];
            mine += k != last && k < vocab;
            last = k;
        }
    }
    uint32_t total;
    const uint32_t before = block_scan<256>(mine, sums, total);
    if (i0 < n && i0 % run == 0)
        starts[i0 / run] = before;
    if (threadIdx.x == 0)
        tiles[blockIdx.x] = total;
}

// Both at once by one workgroup: the starts counted from the first position,
// the tiles' counts 0.
__global__ __launch_bounds__(1024) void embed_starts_small_kernel(const uint32_t *__restrict__ keys,
                                                                  uint32_t n, uint32_t vocab,
                                                                  uint32_t run,
                                                                  uint32_t *__restrict__ starts,
                                                                  uint32_t *__restrict__ tiles,
                                                                  int32_t *__restrict__ count)
{
    __shared__ uint32_t sums[1024 / kWave];
    constexpr uint32_t per = kSmallStarts / 1024u;
    const uint32_t i0 = threadIdx.x * per;
    uint32_t k[per + 1], mine = 0;
#pragma unroll
    for (uint32_t j = 0; j <= per; ++j)   // k[j]: the key before position i0 + j
        k[j] = i0 + j >= 1 && i0 + j <= n ? keys[i0 + j - 1] : 0xFFFFFFFFu;
#pragma unroll
    for (uint32_t j = 0; j < per; ++j)
        mine += k[j + 1] != k[j] && k[j + 1] < vocab;
    uint32_t total;
    const uint32_t before = block_scan<1024>(mine, sums, total);
    if (i0 < n && i0 % run == 0)
        starts[i0 / run] = before;
    if (threadIdx.x < (n + kEmbedTile - 1) / kEmbedTile)
        tiles[threadIdx.x] = 0u;
    if (threadIdx.x == 0)
        *count = (int32_t)total;
}

// In-place exclusive scan of a[0..m) by one workgroup, the total to a[m] (and
// *count).
constexpr uint32_t kScanThreads = 1024, kScanItems = 8;
__global__ __launch_bounds__(kScanThreads) void embed_scan_kernel(uint32_t *__restrict__ a,
                                                                  uint64_t m, int32_t *count)
{
    __shared__ uint32_t sums[kScanThreads / kWave];
    uint32_t carry = 0;
    for (uint64_t c = 0; c < m; c += kScanThreads * kScanItems) {
        const uint64_t i0 = c + (uint64_t)threadIdx.x * kScanItems;
        uint32_t v[kScanItems], mine = 0;
#pragma unroll
        for (uint32_t j = 0; j < kScanItems; ++j) {
            v[j] = i0 + j < m ? a[i0 + j] : 0u;
            mine += v[j];
        }
        uint32_t total, x = carry + block_scan<kScanThreads>(mine, sums, total);
#pragma unroll
        for (uint32_t j = 0; j < kScanItems; ++j) {
            if (i0 + j < m)
                a[i0 + j] = x;
            x += v[j];
        }
        carry += total;
    }
    if (threadIdx.x == 0) {
        a[m] = carry;
        if (count)
            *count = (int32_t)carry;
    }
}

enum class Form { kWrite, kAdd, kRows };

__device__ __forceinline__ uint32_t sum_counts(uint32_t x)
{
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1)
        x += (uint32_t)__shfl_xor((int)x, o, kWave);
    return x;
}

// Segment starts before a tile: scanned, or the sum of up to 64 tiles' counts
// by the wavefront.
__device__ __forceinline__ uint32_t starts_before(const EmbedGrad &e, uint64_t tile)
{
    if (e.scanned)
        return e.tiles[tile];
    const uint32_t lane = threadIdx.x & (kWave - 1);
    return sum_counts(lane < tile ? e.tiles[lane] : 0u);
}

// Zeroes the dense gradient's `rows` rows of `dim` before the sums are written
// over those that are named (one row of all when they lie side by side): a
// workgroup per 4 KiB, one store a lane.  That order of stores reaches 6.85
// TB/s (1 GiB in 157 us), where workgroups of 16 or 64 KiB take 175 or 197 us
// and workgroups that stride through the table 194 to 270.  Zeroing the
// other rows alone, by workgroups behind the sums' own, took 207 us against 175
// for 1000 positions into 65536 x 4096, 52 against 48 for 4001 into 50021 x
// 1001, 23 against 13 for 2000 into 8000 x 512 (each store waited for a search
// of the keys), and 119 against 127 for 65536 into 32000 x 2048.
__global__ __launch_bounds__(256) void embed_zero_kernel(float *out, uint64_t rows, uint64_t dim,
                                                         uint64_t ld, uint64_t vectors)
{
    const uint64_t i = block_number() * 256u + threadIdx.x;   // `vectors` to a row
    const uint64_t row = rows == 1 ? 0 : i / vectors, c = (i - row * vectors) * 4u;
    const vec<float, 4> zero = 0.0f;
    if (row < rows && c < dim)
        store_vec<float, 4>(out + row * ld + c, zero, (int64_t)(dim - c));
}

// Where a finished sum goes; `old` is what is there (kAdd).
template <Form F, int N, bool Nt>
__device__ __forceinline__ void put_row(const EmbedGrad &e, uint64_t row, uint64_t c,
                                        fvec<N> acc, fvec<N> old, int64_t left)
{
    fvec<N> v = acc * e.scale;
    if constexpr (F == Form::kAdd)
        v += old;
    store_vec<float, N, Nt>(e.out + row * e.out_ld + c, v, left);
}

// One pass over g in sorted order.  A wavefront takes a run of e.run sorted
// positions and 256 columns (4 a lane: 16-byte stores; with 8 a lane the sums
// of 16-bit rows went out as pairs of stores 32 bytes apart and took a fifth
// longer).  Keys and positions are the wavefront's own, so they are scalar
// loads and every branch on them is uniform.  A segment inside the run is
// finished here; one that reaches over an end leaves its sum in part[run][0]
// (it began before the run) or part[run][1].
//
// Bound by memory: 65536 x 2048 bf16 into 20000 rows moves 442 MB in 88 us (5.0
// TB/s), 16384 x 4096 bf16 added to a 2 GiB table 364 MB in 67 us (5.4 TB/s);
// a copy of that size reaches 5.4.
// Prefetching the next batch, other batches and longer or shorter runs changed
// nothing.  Nt: the gradient is read and the sums stored non-temporally, from
// 32 MiB of gradient on (the last case, all in all: 102 us, with ordinary
// accesses 110; but 4001 x 1001 float32 into 50021 rows 61 against 58.5, as
// smaller gradients are still in the caches).
template <typename T, Form F, bool Nt>
__global__ __launch_bounds__(256) void embed_grad_kernel(EmbedGrad e, uint32_t cols)
{
    using Scalar = const __attribute__((address_space(4))) uint32_t;
    constexpr int N = 4, U = F == Form::kAdd ? 4 : 8;
    const uint32_t lane = threadIdx.x & (kWave - 1);
    const uint64_t item =
        block_number() * 4u + (uint32_t)__builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    const uint64_t run = item / cols, n = e.n, i0 = run * e.run;
    const uint64_t c = (item % cols * kWave + lane) * N;
    if (i0 >= n)
        return;
    Scalar *keys = (Scalar *)e.keys, *order = (Scalar *)e.order;
    const uint64_t end = n - i0 < e.run ? n : i0 + e.run;
    const int64_t left = c < e.dim ? (int64_t)(e.dim - c) : 0;
    const T *g = (const T *)e.g + c;
    uint64_t seat = 0;
    if constexpr (F == Form::kRows) {
        seat = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane(
                   (int)starts_before(e, i0 / kEmbedTile)) +
               ((Scalar *)e.starts)[run] - 1u;   // of the segment open here
        if (item == 0 && !e.scanned) {
            const uint32_t all = starts_before(e, (n + kEmbedTile - 1) / kEmbedTile);
            if (lane == 0)
                *e.count = (int32_t)all;
        }
    }
    uint32_t last = i0 ? keys[i0 - 1] : 0xFFFFFFFFu;   // the key before
    bool head = last == keys[i0];   // the open segment began before the run
    fvec<N> acc = 0.0f;
    for (uint64_t b = i0; b < end; b += U) {
        uint32_t key[U + 1], pos[U];   // beyond the end: no key at all, 2^32 - 1
#pragma unroll
        for (int j = 0; j <= U; ++j)
            key[j] = b + j < n ? keys[b + j] : 0xFFFFFFFFu;
#pragma unroll
        for (int j = 0; j < U; ++j)
            pos[j] = b + j < n ? order[b + j] : 0u;
        vec<T, N> v[U];
        fvec<N> old[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            v[j] = (T)0.0f;
            old[j] = 0.0f;
            if (key[j] < e.vocab && pos[j] < n) {   // padding is not read
                if (left > 0)
                    v[j] = load_vec<T, N, Nt>(g + pos[j] * e.ld, left);
                if constexpr (F == Form::kAdd)
                    if (key[j] != key[j + 1] && left > 0)
                        old[j] = load_vec<float, N>(e.out + key[j] * e.out_ld + c, left);
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t k = key[j];
            if (k >= e.vocab)
                return;   // padding, or the end: so is everything behind it
            const fvec<N> f = to_f32<T, N>(v[j]);
            if (k != last) {
                acc = f;
                head = false;
                if constexpr (F == Form::kRows) {
                    ++seat;
                    if (c == 0)
                        e.ids[seat] = (int32_t)k;
                }
            } else {
                acc += f;
            }
            last = k;
            if (k != key[j + 1]) {
                if (left > 0) {
                    if (head)
                        store_vec<float, N>(e.part + 2 * run * e.dim + c, acc, left);
                    else
                        put_row<F, N, Nt>(e, F == Form::kRows ? seat : k, c, acc, old[j],
                                          left);
                }
            } else if (b + j + 1 == end && left > 0) {
                store_vec<float, N>(e.part + (2 * run + (head ? 0 : 1)) * e.dim + c, acc, left);
            }
        }
    }
}

// Joins the segments that reach over the end of the run they begin in: part
// 1 of that run, then part 0 of the following ones.  A workgroup looks at 8
// runs and 256 columns.  A segment of at most kJoinShort parts is one
// wavefront's, four columns a lane; a longer one is shared by all 8: 32
// columns each, 8 groups of lanes taking consecutive shares of the parts, whose
// sums are added in a fixed order.  No LDS and no barrier: with the shares
// joined through LDS the short segments slowed down too (16384 positions into
// 131072 x 4096: 115 us against 105).
constexpr uint32_t kJoinThreads = 512, kJoinRuns = 8, kJoinShort = 8, kJoinBatch = 4;
template <Form F>
__global__ __launch_bounds__(kJoinThreads) void embed_join_kernel(EmbedGrad e)
{
    constexpr int N = 4;
    constexpr uint32_t waves = kJoinThreads / kWave;
    const uint32_t lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, R = e.run;
    const uint64_t run0 = (uint64_t)blockIdx.x * kJoinRuns, col0 = (uint64_t)blockIdx.y * 256u;
    // every wavefront: lane l holds the last key of run run0 + l (of this
    // window's runs) and the first key of the one behind it, and whether the
    // run begins a segment that reaches over its end
    uint32_t k0 = 0xFFFFFFFFu, next = 0xFFFFFFFFu, prev = 0xFFFFFFFFu;
    {
        const uint64_t i0 = (run0 + lane) * R, end = i0 + R;
        if (end < e.n) {
            next = e.keys[end];
            if (lane < kJoinRuns) {
                k0 = e.keys[end - 1];
                if (i0)
                    prev = e.keys[i0 - 1];
            }
        }
    }
    const bool joins = k0 < e.vocab && next == k0 && prev != k0;
    uint32_t turn = 0;
    for (uint64_t m = __ballot(joins); m; m &= m - 1, ++turn) {
        const uint32_t q = (uint32_t)__builtin_ctzll(m);
        const uint32_t k = (uint32_t)__shfl((int)k0, (int)q, kWave);
        const uint64_t run = run0 + q;
        // this run and the following ones that begin with k
        const uint64_t stops = ~(__ballot(next == k) >> q);
        uint64_t parts = 1 + (stops ? (uint32_t)__builtin_ctzll(stops) : 64u);
        if (parts == 65 - q) {   // no lane ends it: look at the next 64 runs, and so on
            for (;;) {
                const uint64_t at = (run + parts + lane) * R;
                const uint64_t goes = ~__ballot(at < e.n && e.keys[at] == k);
                parts += goes ? (uint32_t)__builtin_ctzll(goes) : 64u;
                if (goes)
                    break;
            }
        }
        const bool alone = parts <= kJoinShort;
        if (alone && turn % waves != wave)
            continue;
        const uint64_t c = col0 + (alone ? lane * N : wave * 32u + lane % 8u * N);
        const int64_t left = c < e.dim ? (int64_t)(e.dim - c) : 0;
        const uint64_t each = alone ? parts : (parts + 7u) / 8u;
        const uint64_t p0 = alone ? 0 : lane / 8u * each;
        const uint64_t p1 = p0 + each < parts ? p0 + each : parts;
        // what the row's place takes is loaded ahead of the parts
        fvec<N> old = 0.0f;
        uint32_t before = 0, starts = 0, mine = 0, ahead = 0;
        if constexpr (F == Form::kAdd) {
            if (left > 0)
                old = load_vec<float, N>(e.out + (uint64_t)k * e.out_ld + c, left);
        } else if constexpr (F == Form::kRows) {
            const uint64_t tile = run * R / kEmbedTile;
            before = e.scanned ? e.tiles[tile] : lane < tile ? e.tiles[lane] : 0u;
            starts = e.starts[run];
            const uint64_t i = run * R + lane;
            if (lane < R) {
                mine = e.keys[i];
                ahead = i ? e.keys[i - 1] : 0xFFFFFFFFu;
            }
        }
        fvec<N> acc = 0.0f;
        for (uint64_t b = 0; b < each; b += kJoinBatch) {
            vec<float, N> v[kJoinBatch];
#pragma unroll
            for (uint32_t u = 0; u < kJoinBatch; ++u) {
                const uint64_t p = p0 + b + u;
                v[u] = 0.0f;
                if (p < p1 && b + u < each && left > 0)
                    v[u] = load_vec<float, N>(e.part + (2 * (run + p) + (p ? 0 : 1)) * e.dim + c,
                                              left);
            }
#pragma unroll
            for (uint32_t u = 0; u < kJoinBatch; ++u)
                acc += v[u];
        }
        if (!alone) {
#pragma unroll
            for (int o = 8; o < kWave; o <<= 1)
#pragma unroll
                for (int i = 0; i < N; ++i)
                    acc[i] += __shfl_xor(acc[i], o, kWave);
        }
        uint64_t row = k;
        if constexpr (F == Form::kRows) {
            // the last segment that opens in this run
            const uint32_t opens = (uint32_t)__popcll(__ballot(mine != ahead));
            row = (uint64_t)(e.scanned ? before : sum_counts(before)) + starts + opens - 1u;
        }
        if (left > 0 && (alone || lane < 8u))
            put_row<F, N, false>(e, row, c, acc, old, left);
    }
}

uint32_t lanes_for(uint64_t dim, int vec)
{
    const uint64_t want = (dim + vec - 1) / vec;
    uint32_t l = 8;
    while (l < 256 && l < want)
        l *= 2;
    return l;
}

template <typename T, typename O, typename I>
hipError_t lookup(const EmbedTable &t, const void *tokens, uint64_t n, float scale, void *out,
                  uint64_t out_ld, hipStream_t s)
{
    const uint32_t lanes = lanes_for(t.dim, kLookup<T, O>);
    const uint64_t per = 256u / lanes, blocks = (n + per - 1) / per;
    const uint64_t width = (uint64_t)lanes * kLookup<T, O> * kLookupTrips;
    const uint32_t cols = (uint32_t)((t.dim + width - 1) / width);
    const bool two = blocks >= 4096;
    const auto kernel = two ? embed_lookup_kernel<T, O, I, 2> : embed_lookup_kernel<T, O, I, 1>;
    kernel<<<block_grid((two ? (blocks + 1) / 2 : blocks) * cols), 256, 0, s>>>(
        (const T *)t.p, t.vocab, t.dim, t.ld, (const I *)tokens, n, scale, (O *)out, out_ld, lanes,
        cols);
    return hipGetLastError();
}

template <typename T, typename I>
hipError_t lookup(const EmbedTable &t, const void *tokens, uint64_t n, float scale, void *out,
                  int out_type, uint64_t out_ld, hipStream_t s)
{
    switch (out_type) {
    case GCQ_F32: return lookup<T, float, I>(t, tokens, n, scale, out, out_ld, s);
    case GCQ_F16: return lookup<T, _Float16, I>(t, tokens, n, scale, out, out_ld, s);
    default: return lookup<T, __bf16, I>(t, tokens, n, scale, out, out_ld, s);
    }
}

template <typename I>
hipError_t lookup(const EmbedTable &t, const void *tokens, uint64_t n, float scale, void *out,
                  int out_type, uint64_t out_ld, hipStream_t s)
{
    switch (t.type) {
    case GCQ_F32: return lookup<float, I>(t, tokens, n, scale, out, out_type, out_ld, s);
    case GCQ_F16: return lookup<_Float16, I>(t, tokens, n, scale, out, out_type, out_ld, s);
    default: return lookup<__bf16, I>(t, tokens, n, scale, out, out_type, out_ld, s);
    }
}

template <typename I, uint32_t Ti>
void count_sort(const I *tokens, uint32_t n, uint64_t vocab, uint32_t *keys, uint32_t *order,
                hipStream_t s)
{
    const uint32_t groups = 1024u / Ti, share = ((n + groups - 1) / groups + 3u) / 4u * 4u;
    embed_count_sort_kernel<I, Ti><<<(n + Ti - 1) / Ti, 1024, 4 * share * groups, s>>>(
        tokens, n, share, vocab, keys, order);
}

template <typename I, bool First>
void sort_pass(const I *tokens, const uint32_t *keys_in, const uint32_t *order_in, uint32_t n,
               uint64_t vocab, uint32_t shift, uint32_t digit, uint32_t *hist, uint32_t tiles,
               uint32_t *keys_out, uint32_t *order_out, hipStream_t s)
{
    embed_hist_kernel<I, First>
        <<<tiles, kSortThreads, 0, s>>>(tokens, keys_in, n, vocab, shift, digit, hist);
    if (tiles <= kSumTiles) {
        embed_scatter_kernel<I, First, false><<<tiles, kSortThreads, 0, s>>>(
            tokens, keys_in, order_in, n, vocab, shift, digit, hist, tiles, keys_out, order_out);
    } else {
        embed_hist_scan_kernel<<<kBins / kWave, 1024, 0, s>>>(hist, tiles);
        embed_scatter_kernel<I, First, true><<<tiles, kSortThreads, 0, s>>>(
            tokens, keys_in, order_in, n, vocab, shift, digit, hist, tiles, keys_out, order_out);
    }
}

template <typename I>
hipError_t sort_tokens(const I *tokens, uint32_t n, uint64_t vocab, uint32_t *plan, hipStream_t s)
{
    uint32_t *keys[2] = {plan, plan + 2 * (uint64_t)n};
    uint32_t *order[2] = {plan + n, plan + 3 * (uint64_t)n};
    if (n <= kCountSort) {   // a workgroup per CU
        if (n <= 4096)
            count_sort<I, 16>(tokens, n, vocab, keys[0], order[0], s);
        else
            count_sort<I, 32>(tokens, n, vocab, keys[0], order[0], s);
        return hipGetLastError();
    }
    uint32_t bits = 1;
    while (vocab >> bits)   // keys are 0 .. vocab
        ++bits;
    const uint32_t passes = (bits + kDigitBits - 1) / kDigitBits;
    const uint32_t digit = (bits + passes - 1) / passes;
    uint32_t *hist = plan + 4 * (uint64_t)n;
    const uint32_t tiles = (uint32_t)(((uint64_t)n + kSortTile - 1) / kSortTile);
    for (uint32_t p = 0; p < passes; ++p) {
        const uint32_t to = (passes - 1 - p) % 2, from = 1 - to, shift = p * digit;
        if (p == 0)
            sort_pass<I, true>(tokens, nullptr, nullptr, n, vocab, shift, digit, hist, tiles,
                               keys[to], order[to], s);
        else
            sort_pass<I, false>(tokens, keys[from], order[from], n, vocab, shift, digit, hist,
                                tiles, keys[to], order[to], s);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

template <typename T, Form F>
void sum_runs(const EmbedGrad &e, uint64_t runs, hipStream_t s)
{
    const uint32_t cols = (uint32_t)((e.dim + 255) / 256);
    const dim3 grid = block_grid((runs * cols + 3) / 4);
    if (e.n * e.dim * sizeof(T) >= (32ull << 20))
        embed_grad_kernel<T, F, true><<<grid, 256, 0, s>>>(e, cols);
    else
        embed_grad_kernel<T, F, false><<<grid, 256, 0, s>>>(e, cols);
}

template <Form F>
hipError_t grad(EmbedGrad e, hipStream_t s)
{
    const uint64_t runs = (e.n + e.run - 1) / e.run;
    const uint64_t tiles = (e.n + kEmbedTile - 1) / kEmbedTile;
    e.scanned = e.n <= kSmallStarts || tiles > kWave;
    if constexpr (F == Form::kRows) {
        if (runs && e.n <= kSmallStarts) {
            embed_starts_small_kernel<<<1, 1024, 0, s>>>(e.keys, (uint32_t)e.n, (uint32_t)e.vocab,
                                                         e.run, e.starts, e.tiles, e.count);
        } else {
            if (runs)
                embed_starts_kernel<<<(uint32_t)tiles, 256, 0, s>>>(
                    e.keys, (uint32_t)e.n, (uint32_t)e.vocab, e.run, e.starts, e.tiles);
            if (!runs || tiles > kWave)
                embed_scan_kernel<<<1, kScanThreads, 0, s>>>(runs ? e.tiles : (uint32_t *)e.count,
                                                             tiles, runs ? e.count : nullptr);
        }
    }
    if constexpr (F == Form::kWrite) {
        const uint64_t rows = e.out_ld == e.dim ? 1 : e.vocab;
        const uint64_t dim = rows == 1 ? e.vocab * e.dim : e.dim, vectors = (dim + 3) / 4;
        embed_zero_kernel<<<block_grid((rows * vectors + 255) / 256), 256, 0, s>>>(
            e.out, rows, dim, e.out_ld, vectors);
    }
    if (!runs)
        return hipGetLastError();
    switch (e.type) {
    case GCQ_F32: sum_runs<float, F>(e, runs, s); break;
    case GCQ_F16: sum_runs<_Float16, F>(e, runs, s); break;
    default: sum_runs<__bf16, F>(e, runs, s); break;
    }
    if (runs > 1) {
        const dim3 grid((uint32_t)((runs + kJoinRuns - 1) / kJoinRuns),
                        (uint32_t)((e.dim + 4 * kWave - 1) / (4 * kWave)));
        embed_join_kernel<F><<<grid, kJoinThreads, 0, s>>>(e);
    }
    return hipGetLastError();
}

uint64_t up256(uint64_t x) { return (x + 255) / 256 * 256; }

// Sorted positions per run: kEmbedRun, or fewer (8 at least) while the runs
// are too few to give the device 4096 wavefronts of 256 columns.  All positions
// in one run need no join: sorting and summing 20 positions of 512 columns
// takes 16.8 us from the host so, 20.1 with runs of 8 and a join.
constexpr uint64_t kFullWaves = 4096;
constexpr uint32_t kLeastRun = 8;
uint32_t run_length(uint64_t n, uint64_t dim)
{
    uint32_t r = kEmbedRun;
    while (n > kEmbedRun && r > kLeastRun && (n + r - 1) / r * ((dim + 255) / 256) < kFullWaves)
        r /= 2;
    return r;
}

// The workspace's parts: the runs' segment starts, the tiles' counts, two rows
// of open sums a run.
struct WorkLayout {
    uint64_t tiles, part;   // where they begin
};

WorkLayout work_layout(uint64_t n, uint64_t dim)
{
    const uint32_t r = run_length(n, dim);
    const uint64_t runs = (n + r - 1) / r, tiles = (n + kEmbedTile - 1) / kEmbedTile;
    const uint64_t at = up256(4 * runs);
    return {at, at + up256(4 * (tiles + 1))};
}

// The most that any call of up to n positions and dim columns needs, so a
// workspace for the largest batch serves every other one: shorter runs make
// more sums of fewer positions (16000 x 2048 twice as many as 16384 x 2048).
// Runs are shorter than kEmbedRun only while runs twice as long times the
// groups of 256 columns are less than kFullWaves, so there are then less than
// 2 * kFullWaves of runs times groups.
uint64_t most_work(uint64_t n, uint64_t dim)
{
    const uint64_t tiles = (n + kEmbedTile - 1) / kEmbedTile;
    const uint64_t longest = (n + kEmbedRun - 1) / kEmbedRun;
    const uint64_t shortest = n <= kEmbedRun ? longest : (n + kLeastRun - 1) / kLeastRun;
    const uint64_t runs = std::max(longest, std::min(shortest, 2 * kFullWaves));
    const uint64_t sums = std::max(longest * dim, std::min(shortest * dim, 2 * kFullWaves * 256));
    return up256(4 * runs) + up256(4 * (tiles + 1)) + 8 * sums;
}

}  // namespace

uint64_t embed_plan_words(uint64_t n)
{
    const uint64_t tiles = (n + kSortTile - 1) / kSortTile;
    return n <= kCountSort ? 2 * n : 4 * n + (tiles + 1) * kBins;
}

uint64_t embed_work_bytes(uint64_t n, uint64_t dim) { return most_work(n, dim); }

void embed_work_layout(EmbedGrad &e, void *work)
{
    const WorkLayout w = work_layout(e.n, e.dim);
    e.run = run_length(e.n, e.dim);
    e.starts = (uint32_t *)work;
    e.tiles = (uint32_t *)((char *)work + w.tiles);
    e.part = (float *)((char *)work + w.part);
}

hipError_t launch_embed_lookup(const EmbedTable &t, const void *tokens, bool tok64, uint64_t n,
                               float scale, void *out, int out_type, uint64_t out_ld,
                               hipStream_t stream)
{
    return tok64 ? lookup<int64_t>(t, tokens, n, scale, out, out_type, out_ld, stream)
                 : lookup<int32_t>(t, tokens, n, scale, out, out_type, out_ld, stream);
}

hipError_t launch_embed_sort(const void *tokens, bool tok64, uint64_t n, uint64_t vocab,
                             uint32_t *plan, hipStream_t stream)
{
    return tok64 ? sort_tokens((const int64_t *)tokens, (uint32_t)n, vocab, plan, stream)
                 : sort_tokens((const int32_t *)tokens, (uint32_t)n, vocab, plan, stream);
}

hipError_t launch_embed_grad(const EmbedGrad &e, hipStream_t stream)
{
    if (e.count)
        return grad<Form::kRows>(e, stream);
    return e.add ? grad<Form::kAdd>(e, stream) : grad<Form::kWrite>(e, stream);
}

}  // namespace gcq
