// distill.hip -- distillation from a teacher's top logits, loss and
// gradient, for gfx950.
//
// For a row of student logits z[0..V), a temperature T and the teacher's
// entries (index a_j, logit t_j), j < k, of which those with an index outside
// [0, V) count as absent:
//   p = softmax over the entries of t / T       (the top mass, made whole)
//   q = softmax over the vocabulary of z / T,   lse = logsumexp(z / T)
//   loss = s sum_j p_j (log p_j - z[a_j] / T + lse)
//   dz_v = s / T (q_v - sum over j with a_j = v of p_j)
// with s = scale * row_scale.  A row with s = 0 is not read: loss, lse and dz
// are 0.  A row without entries has loss and dz 0.
//
// Sums of exponentials run over exp2((z - m) log2(e) / T) with a running
// maximum m per lane, joined over the lanes: one pass over the row.
// Differences are taken before the factor, whose rounding moves an exponent x
// by 2^-24 x: the largest terms are exact, small ones off by a few of those.
#include "gcq_device.h"
#include "gcq_lm.h"

namespace gcq {

namespace {

using namespace lm;

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLowest = -3.40282347e38f;   // a finite start: -inf - -inf is NaN

// The hardware's exponential, off by about a step; results below 2^-126 may
// come out 0 (a probability that no float32 sum with 1 in it notices).
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// A running maximum m of logits and the sum s of exp2((z - m) * c).
struct Sum {
    float m, s;
};

__device__ __forceinline__ Sum join(Sum a, Sum b, float c)
{
    const float m = fmaxf(a.m, b.m);
    return {m, a.s * exp2_hw((a.m - m) * c) + b.s * exp2_hw((b.m - m) * c)};
}

// Over groups of W neighbouring lanes; each gets the same.
template <int W>
__device__ __forceinline__ Sum join_lanes(Sum a, float c)
{
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
        a = join(a, Sum{__shfl_xor(a.m, o, kWave), __shfl_xor(a.s, o, kWave)}, c);
    return a;
}

// Adds U vectors of logits, the absent ones -inf.
template <int U, int N>
__device__ __forceinline__ void add_logits(Sum &a, const fvec<N> (&z)[U], float c)
{
    float m = a.m;
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < N; ++j)
            m = fmaxf(m, z[u][j]);
    float s = a.s * exp2_hw((a.m - m) * c);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float e[N];
#pragma unroll
        for (int j = 0; j < N; ++j)
            e[j] = exp2_hw((z[u][j] - m) * c);
#pragma unroll
        for (int o = N / 2; o > 0; o >>= 1)
#pragma unroll
            for (int j = 0; j < o; ++j)
                e[j] += e[j + o];
        s += e[0];
    }
    a = {m, s};
}

// Vectors that a lane has in flight: a batch.
constexpr int kFlight = 4;
template <typename T>
using Batch = vec<T, kVec<T>>[kFlight];

// The thread's vectors of a batch at its column `at`, a workgroup's width
// apart, all of them inside the row.
template <typename T, int Threads, bool Nt>
__device__ __forceinline__ void load_batch(Batch<T> &v, const T *z, uint64_t at)
{
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
        v[u] = dev::ld<Nt>((const GCQ_G vec<T, kVec<T>> *)(z + at + u * Threads * kVec<T>));
}

// Where a thread's vectors of a row wait in LDS between two passes.
template <typename T>
using Stash = uint32_t __attribute__((ext_vector_type(4)));
template <typename T>
using Packed = T __attribute__((ext_vector_type(kVec<T>)));

// Keeps the compiler from holding a batch converted to 32 bits, in twice the
// registers, from the first pass to the second.
template <typename T>
__device__ __forceinline__ void hide(Batch<T> &v)
{
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
        Stash<T> x = __builtin_bit_cast(Stash<T>, (Packed<T>)v[u]);
        asm volatile("" : "+v"(x));
        v[u] = __builtin_bit_cast(Packed<T>, x);
    }
}

template <typename T>
__device__ __forceinline__ void add_batch(Sum &a, const Batch<T> &v, float c)
{
    fvec<kVec<T>> f[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
        f[u] = to_f32<T, kVec<T>>(v[u]);
    add_logits<kFlight, kVec<T>>(a, f, c);
}

// dz = value(z) for a batch.  Non-temporal: dz is not read here, so the rows
// still to be read keep the caches.
template <typename T, int Threads, typename F>
__device__ __forceinline__ void put_batch(T *dz, const Batch<T> &v, uint64_t at, F value)
{
    constexpr int N = kVec<T>;
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
        fvec<N> f = to_f32<T, N>(v[u]);
#pragma unroll
        for (int j = 0; j < N; ++j)
            f[j] = value(f[j]);
        dev::st<true>((GCQ_G vec<T, N> *)(dz + at + u * Threads * N), from_f32<T, N>(f));
    }
}

// Non-temporal loads of logits that are read once (Nt): from 96 MiB on they
// pay (2048 x 131072 bf16, loss 80 us against 85, gradient from a kept lse 175
// against 195; at 1024 x 32000, 62 MiB, 15.5 against 15.0 and 29 against 24.5).
constexpr uint64_t kStreamBytes = 96ull << 20;

// Adds columns [c0, c1) of a row, a share of them per thread, and with Keep
// leaves them in the stash.
template <typename T, int Threads, bool Nt, bool Keep = false>
__device__ __forceinline__ void add_row(Sum &a, const T *z, uint64_t c0, uint64_t c1, float c,
                                        Stash<T> *stash = nullptr)
{
    constexpr int N = kVec<T>, U = kFlight;
    constexpr uint64_t step = (uint64_t)Threads * N;
    uint64_t at = c0 + (uint64_t)threadIdx.x * N;
    uint32_t slot = threadIdx.x;
    for (; at + (U - 1) * step + N <= c1; at += U * step) {
        Batch<T> v;
        load_batch<T, Threads, Nt>(v, z, at);
        add_batch<T>(a, v, c);
        if constexpr (Keep) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                stash[slot + u * Threads] = __builtin_bit_cast(Stash<T>, (Packed<T>)v[u]);
            slot += U * Threads;
        }
    }
    for (; at < c1; at += step) {
        const int64_t left = (int64_t)(c1 - at);
        const vec<T, N> v = load_vec<T, N>(z + at, left);
        if constexpr (Keep) {
            stash[slot] = __builtin_bit_cast(Stash<T>, (Packed<T>)v);
            slot += Threads;
        }
        fvec<N> f[1] = {to_f32<T, N>(v)};
#pragma unroll
        for (int j = 0; j < N; ++j)
            f[0][j] = j < left ? f[0][j] : -__builtin_inff();
        add_logits<1, N>(a, f, c);
    }
}

// dz = value(z) over columns [c0, c1), with Kept from the stash.
template <typename T, int Threads, bool Nt, bool Kept = false, typename F>
__device__ __forceinline__ void map_row(const T *z, T *dz, uint64_t c0, uint64_t c1, F value,
                                        const Stash<T> *stash = nullptr)
{
    constexpr int N = kVec<T>, U = kFlight;
    constexpr uint64_t step = (uint64_t)Threads * N;
    uint64_t at = c0 + (uint64_t)threadIdx.x * N;
    uint32_t slot = threadIdx.x;
    for (; at + (U - 1) * step + N <= c1; at += U * step) {
        Batch<T> v;
        if constexpr (Kept) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                v[u] = __builtin_bit_cast(Packed<T>, stash[slot + u * Threads]);
            slot += U * Threads;
        } else {
            load_batch<T, Threads, Nt>(v, z, at);
        }
        put_batch<T, Threads>(dz, v, at, value);
    }
    for (; at < c1; at += step) {
        const int64_t left = (int64_t)(c1 - at);
        vec<T, N> v;
        if constexpr (Kept) {
            v = __builtin_bit_cast(Packed<T>, stash[slot]);
            slot += Threads;
        } else {
            v = load_vec<T, N>(z + at, left);
        }
        fvec<N> f = to_f32<T, N>(v);
#pragma unroll
        for (int j = 0; j < N; ++j)
            f[j] = value(f[j]);
        store_vec<T, N, true>(dz + at, from_f32<T, N>(f), left);
    }
}

template <typename T, int Threads>
__device__ __forceinline__ void zero_row(T *dz, uint64_t c0, uint64_t c1)
{
    constexpr int N = kVec<T>;
    const vec<T, N> zero = (T)0.0f;
    for (uint64_t at = c0 + (uint64_t)threadIdx.x * N; at < c1; at += (uint64_t)Threads * N)
        store_vec<T, N, true>(dz + at, zero, (int64_t)(c1 - at));
}

constexpr uint32_t kNone = 0xFFFFFFFFu;

// LDS of a row's entries, a multiple of 16 bytes.
__host__ __device__ constexpr uint32_t entry_bytes(uint32_t k) { return (12 * k + 15) / 16 * 16; }

template <typename T>
__device__ __forceinline__ float teacher_logit(const Distill &a, uint64_t row, uint32_t j)
{
    if (a.t_f32)
        return ((const GCQ_G float *)a.top)[row * a.top_ld + j];
    return (float)((const GCQ_G T *)a.top)[row * a.top_ld + j];
}

// A teacher's entry: column (kNone: absent), logit (absent: -inf), the
// student's logit there.
struct Entry {
    uint32_t col;
    float top, at;
};

template <typename T>
__device__ __forceinline__ Entry load_entry(const Distill &a, uint64_t row, uint32_t j)
{
    Entry e = {kNone, -__builtin_inff(), 0.0f};
    if (j < a.k) {
        const uint64_t i = row * a.idx_ld + j;
        const uint64_t col = a.idx64 ? (uint64_t)((const GCQ_G int64_t *)a.idx)[i]
                                     : (uint64_t)(int64_t)((const GCQ_G int32_t *)a.idx)[i];
        const float t = teacher_logit<T>(a, row, j);
        if (col < a.vocab) {
            e.col = (uint32_t)col;
            e.top = t;
        }
    }
    return e;
}

// A row's entries: the thread's first in a register (loaded before the row is
// read), those beyond the workgroup's threads in LDS.  Dynamic LDS: k columns,
// k weights and k student's logits.
template <typename T, int Threads>
struct Entries {
    static constexpr int Waves = Threads / kWave;
    uint32_t *col;
    float *w, *z;
    Entry own;

    __device__ __forceinline__ Entries(void *lds, uint32_t k)
        : col((uint32_t *)lds), w((float *)lds + k), z((float *)lds + 2 * k)
    {
    }

    // The student's logits at the entries whose column is in [c0, c1).
    __device__ __forceinline__ void read_logits(const Distill &a, uint64_t row, const T *zr,
                                                uint64_t c0, uint64_t c1)
    {
        const GCQ_G T *p = (const GCQ_G T *)zr;
        if (own.col != kNone && own.col >= c0 && own.col < c1)
            own.at = (float)p[own.col];
        for (uint32_t j = threadIdx.x + Threads; j < a.k; j += Threads) {
            const Entry e = load_entry<T>(a, row, j);
            col[j] = e.col;
            w[j] = e.top;
            z[j] = e.col != kNone && e.col >= c0 && e.col < c1 ? (float)p[e.col] : 0.0f;
        }
    }

    // The thread's largest teacher logit.
    __device__ __forceinline__ float top(const Distill &a) const
    {
        float m = own.top;
        for (uint32_t j = threadIdx.x + Threads; j < a.k; j += Threads)
            m = fmaxf(m, w[j]);
        return m;
    }

    // Turns teacher logits into weights exp((t - m) / T) and adds up the
    // thread's: of w, of w log w and of w (z - zm) / T.
    __device__ __forceinline__ void weigh(const Distill &a, float m, float zm, float (&sum)[3])
    {
        auto one = [&](uint32_t j, float t, float at) {
            const float l = (t - m) / a.temp, e = expf(l);
            if (e != 0.0f) {
                sum[0] += e;
                sum[1] += e * l;
                sum[2] += e * ((at - zm) / a.temp);
            }
            w[j] = e;
        };
        if (threadIdx.x < a.k) {
            col[threadIdx.x] = own.col;
            one(threadIdx.x, own.top, own.at);
        }
        for (uint32_t j = threadIdx.x + Threads; j < a.k; j += Threads)
            one(j, w[j], z[j]);
    }

    // dz at the entries' columns in [c0, c1), over what was stored there
    // before a barrier.  A column named twice loses both probabilities: each
    // of its entries writes the same sum.
    template <typename Q>
    __device__ __forceinline__ void put(const Distill &a, T *dz, uint64_t c0, uint64_t c1, float g,
                                        float sw, Q q) const
    {
        for (uint32_t j = threadIdx.x; j < a.k; j += Threads) {
            const uint32_t cj = col[j];
            if (cj == kNone || cj < c0 || cj >= c1)
                continue;
            float p = 0.0f;
#pragma unroll 4
            for (uint32_t i = 0; i < a.k; ++i)
                p += col[i] == cj ? w[i] : 0.0f;
            ((GCQ_G T *)dz)[cj] = (T)(g * (q(j == threadIdx.x ? own.at : z[j]) - p / sw));
        }
    }
};

// A value per thread -> the workgroup's sum (or maximum), the same for every
// thread; `part` is used by one reduction between two barriers.
template <int Waves, bool Max>
__device__ __forceinline__ void reduce_put(float x, float *part)
{
    x = Max ? max_lanes(x) : sum_lanes(x);
    if ((threadIdx.x & (kWave - 1)) == 0)
        part[threadIdx.x / kWave] = x;
}

template <int Waves, bool Max>
__device__ __forceinline__ float reduce_get(const float *part)
{
    const float x = part[threadIdx.x % Waves];
    return Max ? max_lanes<Waves>(x) : sum_lanes<Waves>(x);
}

// Loss and lse, and with Grad dz too: a workgroup per row.  The entries'
// loads travel while the row is summed.  Both passes together read the row
// twice and write it once, and all of that goes through the fabric between
// the compute units and the last cache (3 GB at 7 TB/s for 4096 x 131072 bf16;
// without the exponentials it took as long).  So each thread keeps its own
// vectors of the row's first columns between the passes: Held batches in
// registers (two workgroups of 512 then fill a compute unit), those up to
// column `kept` in LDS.  Every byte is then moved once: 2.1 GB at 5.1 to 5.3
// TB/s there, where a plain copy of 512 MiB reaches 5.4.  Columns in LDS brought
// 423 -> 393 us, and 65 -> 56 where they are the whole row (8192 x 8000);
// registers beside them nothing more there, but 8192 x 50021 416 -> 374 and
// 2048 x 131072 float32 456 -> 422.
template <typename T, int Threads, int Held, bool Grad, bool Nt>
__global__ __launch_bounds__(Threads, Held ? 4 : 8) void distill_loss_kernel(Distill a,
                                                                             uint64_t kept)
{
    constexpr int Waves = Threads / kWave;
    constexpr uint64_t width = (uint64_t)Threads * kVec<T> * kFlight;
    const uint64_t first = threadIdx.x * kVec<T>;
    extern __shared__ __align__(16) uint32_t lds[];
    __shared__ Sum sum_s[Waves];
    __shared__ float top_s[Waves], red_s[3][Waves];
    const uint32_t tid = threadIdx.x;
    const uint64_t row = block_number();
    if (row >= a.rows)
        return;
    const T *z = (const T *)a.z + row * a.z_ld;
    T *dz = (T *)a.dz + row * a.dz_ld;
    const float s = a.row_scale ? a.scale * a.row_scale[row] : a.scale;
    if (s == 0.0f) {
        if (tid == 0) {
            a.loss[row] = 0.0f;
            a.lse_out[row] = 0.0f;
        }
        if constexpr (Grad)
            zero_row<T, Threads>(dz, 0, a.vocab);
        return;
    }
    Entries<T, Threads> e(lds, a.k);
    e.own = load_entry<T>(a, row, tid);
    const float c = kLog2e / a.temp;
    Sum r = {kLowest, 0.0f};
    Stash<T> *stash = (Stash<T> *)((char *)lds + entry_bytes(a.k));   // [slots][Threads]
    Batch<T> held[Held ? Held : 1];
#pragma unroll
    for (int b = 0; b < Held; ++b)
        load_batch<T, Threads, true>(held[b], z, first + b * width);
#pragma unroll
    for (int b = 0; b < Held; ++b)
        add_batch<T>(r, held[b], c);
    if constexpr (Grad)
        add_row<T, Threads, true, true>(r, z, Held * width, kept, c, stash);
    // the entries' columns have arrived by the row's middle
    constexpr uint64_t step = width / kFlight;
    const uint64_t mid = kept ? kept : a.vocab / (2 * step) * step;
    if (!kept)
        add_row<T, Threads, Nt>(r, z, 0, mid, c);
    e.read_logits(a, row, z, 0, a.vocab);
    add_row<T, Threads, Nt>(r, z, mid, a.vocab, c);
    r = join_lanes<kWave>(r, c);
    if ((tid & (kWave - 1)) == 0)
        sum_s[tid / kWave] = r;
    reduce_put<Waves, true>(e.top(a), top_s);
    __syncthreads();
    r = join_lanes<Waves>(sum_s[tid % Waves], c);
    float tm = reduce_get<Waves, true>(top_s);
    if (tm == -__builtin_inff())
        tm = 0.0f;   // nothing but absent or -inf entries: their sum is 0 (a NaN shows in it)
    float w[3] = {0.0f, 0.0f, 0.0f};
    e.weigh(a, tm, r.m, w);
#pragma unroll
    for (int i = 0; i < 3; ++i)
        reduce_put<Waves, false>(w[i], red_s[i]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 3; ++i)
        w[i] = reduce_get<Waves, false>(red_s[i]);
    const bool any = w[0] != 0.0f;
    if (tid == 0) {
        const float lz = logf(r.s);
        // no finite logit: nothing of q is left where p is
        const float kl = r.s == 0.0f ? __builtin_inff()
                                     : w[1] / w[0] - logf(w[0]) - (w[2] / w[0] - lz);
        a.loss[row] = any ? s * kl : 0.0f;
        a.lse_out[row] = r.m / a.temp + lz;
    }
    if constexpr (Grad) {
        if (!any || r.s == 0.0f) {
            zero_row<T, Threads>(dz, 0, a.vocab);
            return;
        }
        const float g = s / a.temp, inv = 1.0f / r.s, f = g / r.s;
        const auto value = [=](float x) { return exp2_hw((x - r.m) * c) * f; };
#pragma unroll
        for (int b = 0; b < Held; ++b) {
            hide<T>(held[b]);
            put_batch<T, Threads>(dz, held[b], first + b * width, value);
        }
        map_row<T, Threads, true, true>(z, dz, Held * width, kept, value, stash);
        map_row<T, Threads, true>(z, dz, kept, a.vocab, value);
        __syncthreads();
        e.put(a, dz, 0, a.vocab, g, w[0],
              [=](float x) { return exp2_hw((x - r.m) * c) * inv; });
    }
}

// dz from a kept lse; `parts` workgroups share a row, `chunk` columns each.
// The exponent is ((z - hi) - lo) log2(e) / T with hi + lo = lse T, so nothing
// is lost beyond the rounding of lse itself to float32: q is off by up to
// 2^-24 |lse| relative, and a row's gradient sums to that instead of 0.
// Whether the row has entries at all is known only after
// the dense pass; a row without is zeroed then.  Bound by memory: 4096 x 131072
// bf16 336 us (2.1 GB, 6.2 TB/s).
template <typename T, int Threads, bool Nt>
__global__ __launch_bounds__(Threads) void distill_grad_kernel(Distill a, uint64_t parts,
                                                               uint64_t chunk)
{
    constexpr int Waves = Threads / kWave;
    extern __shared__ __align__(16) uint32_t lds[];
    __shared__ float top_s[Waves], red_s[Waves];
    const uint64_t row = block_number() / parts, c0 = block_number() % parts * chunk;
    if (row >= a.rows)
        return;
    const uint64_t c1 = c0 + chunk < a.vocab ? c0 + chunk : a.vocab;
    const T *z = (const T *)a.z + row * a.z_ld;
    T *dz = (T *)a.dz + row * a.dz_ld;
    const float s = a.row_scale ? a.scale * a.row_scale[row] : a.scale;
    const float lse = a.lse[row];
    if (s == 0.0f || lse == -__builtin_inff()) {
        zero_row<T, Threads>(dz, c0, c1);
        return;
    }
    Entries<T, Threads> e(lds, a.k);
    e.own = load_entry<T>(a, row, threadIdx.x);
    e.read_logits(a, row, z, c0, c1);
    if (a.dz == a.z)
        __syncthreads();   // in place: they are read before any is written
    const float c = kLog2e / a.temp, g = s / a.temp;
    const float hi = lse * a.temp, lo = fmaf(lse, a.temp, -hi);
    const auto q = [=](float x) { return exp2_hw(((x - hi) - lo) * c); };
    map_row<T, Threads, Nt>(z, dz, c0, c1, [=](float x) { return q(x) * g; });
    reduce_put<Waves, true>(e.top(a), top_s);
    __syncthreads();
    float tm = reduce_get<Waves, true>(top_s);
    if (tm == -__builtin_inff())
        tm = 0.0f;
    float w[3] = {0.0f, 0.0f, 0.0f};
    e.weigh(a, tm, 0.0f, w);
    reduce_put<Waves, false>(w[0], red_s);
    __syncthreads();
    const float sw = reduce_get<Waves, false>(red_s);
    if (sw == 0.0f)
        zero_row<T, Threads>(dz, c0, c1);
    else
        e.put(a, dz, c0, c1, g, sw, q);
}

template <typename T, int Threads>
void loss(const Distill &a, hipStream_t s)
{
    const auto kernel = a.rows * a.vocab * sizeof(T) >= kStreamBytes
                            ? distill_loss_kernel<T, Threads, 0, false, true>
                            : distill_loss_kernel<T, Threads, 0, false, false>;
    kernel<<<block_grid(a.rows), Threads, entry_bytes(a.k), s>>>(a, 0);
}

// Rows of at least Held batches.
template <typename T, int Threads, int Held>
void loss_grad(const Distill &a, hipStream_t s)
{
    // vectors a thread that fit the workgroup's share of a compute unit's LDS
    constexpr uint64_t step = (uint64_t)Threads * kVec<T>, held = Held * kFlight * step;
    constexpr uint32_t waves = Held ? 16 : 32, slot = Threads * 16;
    constexpr uint32_t share = dev::kLdsBytesPerCu / (waves * kWave / Threads) - 512u;
    const uint32_t lds = entry_bytes(a.k);
    const uint64_t room = held + (lds < share ? (share - lds) / slot : 0) * step;
    const uint64_t kept = a.vocab < room ? a.vocab : room;
    const uint32_t slots = (uint32_t)((kept - held + step - 1) / step);
    distill_loss_kernel<T, Threads, Held, true, false>
        <<<block_grid(a.rows), Threads, lds + slots * slot, s>>>(a, kept);
}

template <typename T>
hipError_t loss(const Distill &a, hipStream_t s)
{
    // A workgroup for a few vectors a lane.  Long rows get few, large
    // workgroups: with many rows in flight at once they no longer stay on the
    // chip between the two passes.  Loss and gradient in bf16, us with 64 / 256
    // / 512 / 1024 threads, the columns that fit in LDS and none in registers:
    // 8192 x 1000 21 / 34 / 60 / 146; 8192 x 8000 73 / 66 / 90 / 169; 8192 x
    // 32000 270 / 225 / 209 / 260; 4096 x 60000 274 / 233 / 218 / 207.  Batches
    // in registers too: 8192 x 16000 with 256 threads 111 with one, 122 without;
    // with 512 threads 8192 x 40000 261 with two, 259 without; 8192 x 50021 374
    // with three, 416 without; 4096 x 100000 313 with four, 328 with three; 4096
    // x 131072 402 with four, 438 without (1024 threads 396, but 2048 x 131072
    // float32 445 against 422).  The loss alone with 64 / 256 / 512 / 1024: 8192
    // x 1000 11 / 22 / 42 / 91; 8192 x 8000 29 / 39 / 53 / 95, but 128 x 32000
    // 16 / 9.6 / 9.5 / 9.3; 4096 x 131072 162 / 157 / 155 / 150.
    const uint64_t bytes = a.vocab * sizeof(T);
    if (bytes <= 8192)
        a.dz ? loss_grad<T, 64, 0>(a, s) : loss<T, 64>(a, s);
    else if (bytes <= 32768)
        !a.dz             ? loss<T, 256>(a, s)
        : bytes >= 16384  ? loss_grad<T, 256, 1>(a, s)
                          : loss_grad<T, 256, 0>(a, s);
    else if (bytes <= 98304)
        a.dz ? loss_grad<T, 512, 0>(a, s) : loss<T, 512>(a, s);
    else
        !a.dz             ? loss<T, 1024>(a, s)
        : bytes >= 131072 ? loss_grad<T, 512, 4>(a, s)
                          : loss_grad<T, 512, 3>(a, s);
    return hipGetLastError();
}

template <typename T>
hipError_t grad(const Distill &a, hipStream_t s)
{
    // one batch a lane: 1021 x 50021 float32 74 us, with two 83, with half of
    // one 72; 4096 x 131072 bf16 336, 353, 361
    constexpr int threads = 256;
    const uint64_t chunk = (uint64_t)threads * kVec<T> * kFlight;
    const uint64_t parts = (a.vocab + chunk - 1) / chunk;
    const auto kernel = a.rows * a.vocab * sizeof(T) >= kStreamBytes
                            ? distill_grad_kernel<T, threads, true>
                            : distill_grad_kernel<T, threads, false>;
    kernel<<<block_grid(a.rows * parts), threads, entry_bytes(a.k), s>>>(a, parts, chunk);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_distill(const Distill &a, hipStream_t stream)
{
    switch (a.type) {
    case GCQ_F32: return a.lse ? grad<float>(a, stream) : loss<float>(a, stream);
    case GCQ_F16: return a.lse ? grad<_Float16>(a, stream) : loss<_Float16>(a, stream);
    default: return a.lse ? grad<__bf16>(a, stream) : loss<__bf16>(a, stream);
    }
}

}  // namespace gcq
