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
#include "gcq_device.h"
#include "gcq_lm.h"

namespace gcq {

namespace {

using namespace lm;

// ------------------------------------------------------------------ lookup
// L lanes share a row (a power of two up to 256), so a workgroup of 256
// threads copies 256 / L rows at once; a lane strides over its row.
template <typename T, typename O, typename I>
__global__ __launch_bounds__(256) void embed_lookup_kernel(const T *__restrict__ table,
                                                           uint64_t vocab, uint64_t dim,
                                                           uint64_t ld,
                                                           const I *__restrict__ tokens,
                                                           uint64_t n, float scale,
                                                           O *__restrict__ out, uint64_t out_ld,
                                                           uint32_t lanes)
{
    constexpr int N = kVec<T>;
    const uint32_t lane = threadIdx.x & (lanes - 1), slot = threadIdx.x / lanes;
    const uint64_t row = block_number() * (256u / lanes) + slot;
    if (row >= n)
        return;
    const uint64_t tok = (uint64_t)(int64_t)((const GCQ_G I *)tokens)[row];
    const bool real = tok < vocab;   // a negative token is past any vocab
    const T *src = table + (real ? tok : 0) * ld;
    O *dst = out + row * out_ld;
#pragma unroll 2
    for (uint64_t c = (uint64_t)lane * N; c < dim; c += (uint64_t)lanes * N) {
        const int64_t left = (int64_t)(dim - c);
        fvec<N> f = 0.0f;
        if (real)
            f = to_f32<T, N>(load_vec<T, N>(src + c, left)) * scale;
        store_vec<O, N>(dst + c, from_f32<O, N>(f), left);
    }
}

// -------------------------------------------------------------------- sort
// Least-significant-digit radix sort of (token, position), digits of at most
// 9 bits, tiles of 2048 positions.  A wavefront ranks 64 tokens at a time:
// a ballot per digit bit gives each lane the lanes that share its digit, so
// the rank is a count of lower lanes plus the wavefront's count so far, and
// equal digits keep their order.
constexpr uint32_t kDigitBits = 9, kBins = 1u << kDigitBits;
constexpr uint32_t kSortThreads = 256, kSortItems = 8;
constexpr uint32_t kSortTile = kSortThreads * kSortItems;
// One workgroup sorts this many in LDS, in one launch.
constexpr uint32_t kSmallThreads = 1024, kSmallItems = 4;
constexpr uint32_t kSmallSort = kSmallThreads * kSmallItems;

template <typename I>
__device__ __forceinline__ uint32_t token_key(const I *tokens, uint64_t i, uint64_t vocab)
{
    const uint64_t t = (uint64_t)(int64_t)((const GCQ_G I *)tokens)[i];
    return (uint32_t)(t < vocab ? t : vocab);   // padding sorts behind every token
}

__device__ __forceinline__ void wave_order()
{
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Ranks this wavefront's Items digits among its earlier ones of equal value;
// cnt[bin] (zero on entry) ends as the wavefront's histogram.  Items with
// digit >= kBins take no part.
template <int Items, typename C>
__device__ __forceinline__ void wave_rank(const uint32_t (&digit)[Items], uint32_t bits, C *cnt,
                                          uint32_t (&rank)[Items])
{
    const uint32_t lane = threadIdx.x & (kWave - 1);
    const uint64_t below = (1ull << lane) - 1u;
#pragma unroll
    for (int j = 0; j < Items; ++j) {
        const bool in = digit[j] < kBins;
        uint64_t peers = __ballot(in);
        for (uint32_t b = 0; b < bits; ++b) {
            const bool one = (digit[j] >> b) & 1u;
            const uint64_t m = __ballot(one);
            peers &= one ? m : ~m;
        }
        uint32_t first = 0;
        if (in)
            first = cnt[digit[j]];
        wave_order();   // every lane has read before the count moves
        if (in && (peers & below) == 0)
            cnt[digit[j]] = (C)(first + (uint32_t)__popcll(peers));
        wave_order();
        rank[j] = first + (uint32_t)__popcll(peers & below);
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

template <typename I>
__global__ __launch_bounds__(kSmallThreads) void embed_sort_small_kernel(
    const I *__restrict__ tokens, uint32_t n, uint64_t vocab, uint32_t bits, uint32_t digit_bits,
    uint32_t *__restrict__ keys, uint32_t *__restrict__ order)
{
    constexpr uint32_t waves = kSmallThreads / kWave;
    __shared__ uint32_t key_s[kSmallSort];
    __shared__ uint16_t pos_s[kSmallSort];
    __shared__ uint16_t cnt[waves][kBins];
    __shared__ uint32_t base[kBins], sums[waves];
    const uint32_t tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const uint32_t at = wave * kWave * kSmallItems + lane;   // item j: at + 64 j
    uint32_t key[kSmallItems], pos[kSmallItems], rank[kSmallItems], digit[kSmallItems];
#pragma unroll
    for (uint32_t j = 0; j < kSmallItems; ++j) {
        pos[j] = at + kWave * j;
        key[j] = pos[j] < n ? token_key(tokens, pos[j], vocab) : 0u;
    }
    for (uint32_t shift = 0; shift < bits; shift += digit_bits) {
        for (uint32_t i = tid; i < waves * kBins; i += kSmallThreads)
            (&cnt[0][0])[i] = 0;
        __syncthreads();
        const uint32_t mask = (1u << digit_bits) - 1u;
#pragma unroll
        for (uint32_t j = 0; j < kSmallItems; ++j)
            digit[j] = at + kWave * j < n ? (key[j] >> shift) & mask : kBins;
        wave_rank<kSmallItems>(digit, digit_bits, cnt[wave], rank);
        __syncthreads();
        uint32_t mine = 0;   // bin tid: this workgroup's count, each wavefront's start
        if (tid < kBins) {
            for (uint32_t w = 0; w < waves; ++w) {
                const uint32_t c = cnt[w][tid];
                cnt[w][tid] = (uint16_t)mine;
                mine += c;
            }
        }
        uint32_t total;
        const uint32_t first = block_scan<kSmallThreads>(mine, sums, total);
        if (tid < kBins)
            base[tid] = first;
        __syncthreads();
#pragma unroll
        for (uint32_t j = 0; j < kSmallItems; ++j) {
            if (digit[j] < kBins) {
                const uint32_t to = base[digit[j]] + cnt[wave][digit[j]] + rank[j];
                key_s[to] = key[j];
                pos_s[to] = (uint16_t)pos[j];
            }
        }
        __syncthreads();
#pragma unroll
        for (uint32_t j = 0; j < kSmallItems; ++j) {
            const uint32_t i = at + kWave * j;
            if (i < n) {
                key[j] = key_s[i];
                pos[j] = pos_s[i];
            }
        }
        // the next pass's barriers come between these reads and its writes
    }
#pragma unroll
    for (uint32_t j = 0; j < kSmallItems; ++j) {
        const uint32_t i = at + kWave * j;
        if (i < n) {
            keys[i] = key[j];
            order[i] = pos[j];
        }
    }
}

// The tile's digit counts, digit-major: hist[digit * tiles + tile].
// First: keys come from the tokens.
template <typename I, bool First>
__global__ __launch_bounds__(kSortThreads) void embed_hist_kernel(
    const I *__restrict__ tokens, const uint32_t *__restrict__ keys, uint32_t n, uint64_t vocab,
    uint32_t shift, uint32_t digit_bits, uint32_t *__restrict__ hist, uint32_t tiles)
{
    __shared__ uint32_t cnt[kBins];
    const uint32_t bins = 1u << digit_bits, tid = threadIdx.x;
    for (uint32_t i = tid; i < bins; i += kSortThreads)
        cnt[i] = 0;
    __syncthreads();
    const uint64_t t0 = (uint64_t)blockIdx.x * kSortTile;
#pragma unroll
    for (uint32_t j = 0; j < kSortItems; ++j) {
        const uint64_t i = t0 + tid + kSortThreads * j;
        if (i < n) {
            const uint32_t k = First ? token_key(tokens, i, vocab) : keys[i];
            atomicAdd(&cnt[(k >> shift) & (bins - 1u)], 1u);   // whole numbers: any order
        }
    }
    __syncthreads();
    for (uint32_t i = tid; i < bins; i += kSortThreads)
        hist[(uint64_t)i * tiles + blockIdx.x] = cnt[i];
}

// In-place exclusive scan of a[0..m) by one workgroup, the total to a[m] if
// `put_total`.
constexpr uint32_t kScanThreads = 1024, kScanItems = 8;
__global__ __launch_bounds__(kScanThreads) void embed_scan_kernel(uint32_t *__restrict__ a,
                                                                  uint64_t m, bool put_total)
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
    if (put_total && threadIdx.x == 0)
        a[m] = carry;
}

template <typename I, bool First>
__global__ __launch_bounds__(kSortThreads) void embed_scatter_kernel(
    const I *__restrict__ tokens, const uint32_t *__restrict__ keys_in,
    const uint32_t *__restrict__ order_in, uint32_t n, uint64_t vocab, uint32_t shift,
    uint32_t digit_bits, const uint32_t *__restrict__ hist, uint32_t tiles,
    uint32_t *__restrict__ keys_out, uint32_t *__restrict__ order_out)
{
    constexpr uint32_t waves = kSortThreads / kWave;
    __shared__ uint32_t cnt[waves][kBins];
    const uint32_t bins = 1u << digit_bits, tid = threadIdx.x;
    const uint32_t lane = tid & (kWave - 1), wave = tid / kWave;
    for (uint32_t i = tid; i < waves * kBins; i += kSortThreads)
        (&cnt[0][0])[i] = 0;
    __syncthreads();
    const uint64_t at = (uint64_t)blockIdx.x * kSortTile + wave * kWave * kSortItems + lane;
    uint32_t key[kSortItems], pos[kSortItems], rank[kSortItems], digit[kSortItems];
#pragma unroll
    for (uint32_t j = 0; j < kSortItems; ++j) {
        const uint64_t i = at + kWave * j;
        key[j] = 0;
        pos[j] = (uint32_t)i;
        if (i < n) {
            key[j] = First ? token_key(tokens, i, vocab) : keys_in[i];
            if (!First)
                pos[j] = order_in[i];
        }
        digit[j] = i < n ? (key[j] >> shift) & (bins - 1u) : kBins;
    }
    wave_rank<kSortItems>(digit, digit_bits, cnt[wave], rank);
    __syncthreads();
    for (uint32_t b = tid; b < bins; b += kSortThreads) {
        uint32_t first = hist[(uint64_t)b * tiles + blockIdx.x];
        for (uint32_t w = 0; w < waves; ++w) {
            const uint32_t c = cnt[w][b];
            cnt[w][b] = first;
            first += c;
        }
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
// Segment starts before each run of kEmbedRun sorted positions (within its
// tile), and each tile's count.
__global__ __launch_bounds__(256) void embed_starts_kernel(const uint32_t *__restrict__ keys,
                                                           uint32_t n, uint32_t vocab,
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
    if (i0 < n && i0 % kEmbedRun == 0)
        starts[i0 / kEmbedRun] = before;
    if (threadIdx.x == 0)
        tiles[blockIdx.x] = total;
}

enum class Form { kWrite, kAdd, kRows };

// Where a finished sum goes.
template <Form F, int N>
__device__ __forceinline__ void put_row(const EmbedGrad &e, uint64_t row, uint64_t c,
                                        fvec<N> acc, int64_t left)
{
    float *p = e.out + row * e.out_ld + c;
    fvec<N> v = acc * e.scale;
    if constexpr (F == Form::kAdd)
        v += load_vec<float, N>(p, left);
    store_vec<float, N>(p, v, left);
}

// One pass over g in sorted order.  L lanes (a power of two up to 256) share
// a run of 32 sorted positions and L * N columns.  A segment inside the run
// is finished here; one that reaches over an end leaves its sum in
// part[run][0] (it began before the run) or part[run][1].
template <typename T, Form F>
__global__ __launch_bounds__(256) void embed_grad_kernel(EmbedGrad e, uint32_t lanes)
{
    constexpr int N = kVec<T>, U = 8;
    __shared__ uint32_t key_s[32][kEmbedRun + 2], pos_s[32][kEmbedRun];
    const uint32_t groups = 256u / lanes, lane = threadIdx.x & (lanes - 1);
    const uint32_t slot = threadIdx.x / lanes;
    const uint64_t run0 = (uint64_t)blockIdx.x * groups;
    const uint64_t n = e.n;
    // key_s[s][1 + i]: the run's keys, with one neighbour on each side
    // (beyond the ends: no key at all, 2^32 - 1)
    for (uint32_t i = threadIdx.x; i < groups * (kEmbedRun + 2); i += 256u) {
        const uint32_t s = i / (kEmbedRun + 2), j = i % (kEmbedRun + 2);
        const uint64_t at = (run0 + s) * kEmbedRun + j;   // one past the position
        key_s[s][j] = at >= 1 && at <= n ? e.keys[at - 1] : 0xFFFFFFFFu;
        if (j < kEmbedRun && at < n)
            pos_s[s][j] = e.order[at];
    }
    __syncthreads();
    const uint64_t run = run0 + slot, i0 = run * kEmbedRun;
    const uint64_t c = ((uint64_t)blockIdx.y * lanes + lane) * N;
    if (i0 >= n || c >= e.dim)
        return;
    const uint32_t len = n - i0 < kEmbedRun ? (uint32_t)(n - i0) : kEmbedRun;
    const uint32_t *key = key_s[slot] + 1;
    const int64_t left = (int64_t)(e.dim - c);
    const T *g = (const T *)e.g + c;
    uint64_t seat = 0;
    if constexpr (F == Form::kRows)
        seat = (uint64_t)e.tiles[i0 / kEmbedTile] + e.starts[run] - 1u;   // of the segment open here
    fvec<N> acc = 0.0f;
    for (uint32_t b = 0; b < len; b += U) {
        vec<T, N> v[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            v[j] = (T)0.0f;
            if (b + j < len && key[b + j] < e.vocab) {
                const uint64_t at = pos_s[slot][b + j];
                if (at < n)
                    v[j] = load_vec<T, N>(g + at * e.ld, left);
            }
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const uint32_t i = b + j;
            if (i >= len)
                break;
            const uint32_t k = key[i];
            if (k >= e.vocab)
                break;   // padding: so is everything behind it
            const bool opens = k != key_s[slot][i];
            if constexpr (F == Form::kRows) {
                if (opens) {
                    ++seat;
                    if (c == 0)
                        e.ids[seat] = (int32_t)k;
                }
            }
            const fvec<N> f = to_f32<T, N>(v[j]);
            acc = opens || i == 0 ? f : acc + f;
            const bool closes = k != key[i + 1];
            if (!closes && i + 1 < len)
                continue;
            // did this segment begin before the run?
            const bool head = key[0] == k && key_s[slot][0] == k;
            if (closes && !head) {
                put_row<F, N>(e, F == Form::kRows ? seat : k, c, acc, left);
            } else {
                float *p = e.part + (2 * run + (head ? 0 : 1)) * e.dim + c;
                store_vec<float, N>(p, acc, left);
            }
        }
    }
    if constexpr (F == Form::kRows) {
        if (i0 == 0 && c == 0)
            *e.count = (int32_t)e.tiles[(n + kEmbedTile - 1) / kEmbedTile];
    }
}

// Joins the segments that reach over the end of the run they begin in: part
// 1 of that run, then part 0 of the following ones, summed by 8 wavefronts
// over consecutive shares and the shares in order.
constexpr uint32_t kJoinThreads = 512, kJoinRuns = 4;
template <Form F>
__global__ __launch_bounds__(kJoinThreads) void embed_join_kernel(EmbedGrad e, uint32_t runs)
{
    constexpr int N = 4;
    constexpr uint32_t waves = kJoinThreads / kWave;
    __shared__ fvec<N> share[waves][kWave];
    const uint32_t lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const uint64_t c = ((uint64_t)blockIdx.y * kWave + lane) * N;
    const int64_t left = c < e.dim ? (int64_t)(e.dim - c) : 0;
    for (uint32_t q = 0; q < kJoinRuns; ++q) {
        const uint64_t run = (uint64_t)blockIdx.x * kJoinRuns + q;
        const uint64_t i0 = run * kEmbedRun, end = i0 + kEmbedRun;
        if (run >= runs || end >= e.n)
            return;
        const uint32_t k = e.keys[end - 1];
        if (k >= e.vocab || k != e.keys[end])
            continue;   // nothing reaches over
        if (i0 && e.keys[i0 - 1] == k)
            continue;   // it began earlier: an earlier run joins it
        uint64_t lo = end, hi = e.n;   // the first position behind the segment
        while (lo < hi) {
            const uint64_t mid = (lo + hi) / 2;
            if (e.keys[mid] == k)
                lo = mid + 1;
            else
                hi = mid;
        }
        const uint64_t parts = (lo - 1) / kEmbedRun - run + 1;   // runs it touches
        const uint64_t each = (parts + waves - 1) / waves;
        const uint64_t p0 = wave * each, p1 = p0 + each < parts ? p0 + each : parts;
        fvec<N> acc = 0.0f;
        if (left > 0) {
#pragma unroll 8
            for (uint64_t p = p0; p < p1; ++p)
                acc += load_vec<float, N>(e.part + (2 * (run + p) + (p ? 0 : 1)) * e.dim + c, left);
        }
        share[wave][lane] = acc;
        __syncthreads();
        if (wave == 0 && left > 0) {
            for (uint32_t w = 1; w < waves && w * each < parts; ++w)
                acc += share[w][lane];
            uint64_t row = k;
            if constexpr (F == Form::kRows) {
                // the last segment that opens in this run
                uint32_t opens = 0;
                for (uint32_t i = 0; i < kEmbedRun; ++i)
                    opens += i0 + i == 0 || e.keys[i0 + i] != e.keys[i0 + i - 1];
                row = (uint64_t)e.tiles[i0 / kEmbedTile] + e.starts[run] + opens - 1u;
            }
            put_row<F, N>(e, row, c, acc, left);
        }
        __syncthreads();
    }
}

// Zeroes the rows of the dense gradient that no position names: 64 rows per
// workgroup, one lane each looks its row up in the sorted tokens.
__global__ __launch_bounds__(256) void embed_zero_kernel(EmbedGrad e)
{
    __shared__ uint64_t untouched;
    const uint64_t v0 = block_number() * kWave;
    if (threadIdx.x < kWave) {
        const uint64_t v = v0 + threadIdx.x;
        uint64_t lo = 0, hi = e.n;
        while (lo < hi) {
            const uint64_t mid = (lo + hi) / 2;
            if (e.keys[mid] < v)
                lo = mid + 1;
            else
                hi = mid;
        }
        const uint64_t m = __ballot(v < e.vocab && !(lo < e.n && e.keys[lo] == v));
        if (threadIdx.x == 0)
            untouched = m;
    }
    __syncthreads();
    const vec<float, 4> zero = 0.0f;
    for (uint64_t m = untouched; m; m &= m - 1) {
        float *row = e.out + (v0 + (uint64_t)__builtin_ctzll(m)) * e.out_ld;
        for (uint64_t c = threadIdx.x * 4u; c < e.dim; c += 1024u)
            store_vec<float, 4>(row + c, zero, (int64_t)(e.dim - c));
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
    const uint32_t lanes = lanes_for(t.dim, kVec<T>);
    const uint64_t per = 256u / lanes;
    embed_lookup_kernel<T, O, I><<<block_grid((n + per - 1) / per), 256, 0, s>>>(
        (const T *)t.p, t.vocab, t.dim, t.ld, (const I *)tokens, n, scale, (O *)out, out_ld, lanes);
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

template <typename I>
hipError_t sort_tokens(const I *tokens, uint32_t n, uint64_t vocab, uint32_t *plan, hipStream_t s)
{
    uint32_t bits = 1;
    while (vocab >> bits)   // keys are 0 .. vocab
        ++bits;
    const uint32_t passes = (bits + kDigitBits - 1) / kDigitBits;
    const uint32_t digit = (bits + passes - 1) / passes;
    uint32_t *keys[2] = {plan, plan + 2 * (uint64_t)n};
    uint32_t *order[2] = {plan + n, plan + 3 * (uint64_t)n};
    if (n <= kSmallSort) {
        embed_sort_small_kernel<I>
            <<<1, kSmallThreads, 0, s>>>(tokens, n, vocab, bits, digit, keys[0], order[0]);
        return hipGetLastError();
    }
    uint32_t *hist = plan + 4 * (uint64_t)n;
    const uint32_t tiles = (uint32_t)(((uint64_t)n + kSortTile - 1) / kSortTile);
    for (uint32_t p = 0; p < passes; ++p) {
        const uint32_t to = (passes - 1 - p) % 2, from = 1 - to, shift = p * digit;
        if (p == 0)
            embed_hist_kernel<I, true><<<tiles, kSortThreads, 0, s>>>(
                tokens, nullptr, n, vocab, shift, digit, hist, tiles);
        else
            embed_hist_kernel<I, false><<<tiles, kSortThreads, 0, s>>>(
                tokens, keys[from], n, vocab, shift, digit, hist, tiles);
        embed_scan_kernel<<<1, kScanThreads, 0, s>>>(hist, (uint64_t)tiles << digit, false);
        if (p == 0)
            embed_scatter_kernel<I, true><<<tiles, kSortThreads, 0, s>>>(
                tokens, nullptr, nullptr, n, vocab, shift, digit, hist, tiles, keys[to], order[to]);
        else
            embed_scatter_kernel<I, false><<<tiles, kSortThreads, 0, s>>>(
                tokens, keys[from], order[from], n, vocab, shift, digit, hist, tiles, keys[to],
                order[to]);
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

template <Form F>
hipError_t grad(const EmbedGrad &e, hipStream_t s)
{
    const uint64_t runs = (e.n + kEmbedRun - 1) / kEmbedRun;
    if (F == Form::kRows && !runs)
        embed_scan_kernel<<<1, kScanThreads, 0, s>>>((uint32_t *)e.count, 0, true);
    if constexpr (F == Form::kWrite)
        embed_zero_kernel<<<block_grid((e.vocab + kWave - 1) / kWave), 256, 0, s>>>(e);
    if (!runs)
        return hipGetLastError();
    if constexpr (F == Form::kRows) {
        const uint64_t tiles = (e.n + kEmbedTile - 1) / kEmbedTile;
        embed_starts_kernel<<<(uint32_t)tiles, 256, 0, s>>>(e.keys, (uint32_t)e.n,
                                                            (uint32_t)e.vocab, e.starts, e.tiles);
        embed_scan_kernel<<<1, kScanThreads, 0, s>>>(e.tiles, tiles, true);
    }
    const int vec = e.type == GCQ_F32 ? kVec<float> : kVec<_Float16>;
    const uint32_t lanes = lanes_for(e.dim, vec), groups = 256u / lanes;
    const uint64_t cols = (e.dim + (uint64_t)lanes * vec - 1) / ((uint64_t)lanes * vec);
    const dim3 grid((uint32_t)((runs + groups - 1) / groups), (uint32_t)cols);
    switch (e.type) {
    case GCQ_F32: embed_grad_kernel<float, F><<<grid, 256, 0, s>>>(e, lanes); break;
    case GCQ_F16: embed_grad_kernel<_Float16, F><<<grid, 256, 0, s>>>(e, lanes); break;
    default: embed_grad_kernel<__bf16, F><<<grid, 256, 0, s>>>(e, lanes); break;
    }
    if (runs > 1) {
        const dim3 jgrid((uint32_t)((runs + kJoinRuns - 1) / kJoinRuns),
                         (uint32_t)((e.dim + 4 * kWave - 1) / (4 * kWave)));
        embed_join_kernel<F><<<jgrid, kJoinThreads, 0, s>>>(e, (uint32_t)runs);
    }
    return hipGetLastError();
}

uint64_t up256(uint64_t x) { return (x + 255) / 256 * 256; }

}  // namespace

uint64_t embed_plan_words(uint64_t n)
{
    const uint64_t tiles = (n + kSortTile - 1) / kSortTile;
    return 4 * n + (n > kSmallSort ? tiles * kBins : 0);
}

uint64_t embed_work_bytes(uint64_t n, uint64_t dim)
{
    const uint64_t runs = (n + kEmbedRun - 1) / kEmbedRun;
    const uint64_t tiles = (n + kEmbedTile - 1) / kEmbedTile;
    return up256(4 * runs) + up256(4 * (tiles + 1)) + 8 * runs * dim;
}

void embed_work_layout(EmbedGrad &e, void *work)
{
    const uint64_t runs = (e.n + kEmbedRun - 1) / kEmbedRun;
    const uint64_t tiles = (e.n + kEmbedTile - 1) / kEmbedTile;
    char *p = (char *)work;
    e.starts = (uint32_t *)p;
    e.tiles = (uint32_t *)(p + up256(4 * runs));
    e.part = (float *)(p + up256(4 * runs) + up256(4 * (tiles + 1)));
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
