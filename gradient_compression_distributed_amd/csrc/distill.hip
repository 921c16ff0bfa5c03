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
// Differences are taken before the factor, so the largest terms are exact.
#include "gcq_device.h"
#include "gcq_lm.h"

namespace gcq {

namespace {

using namespace lm;

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLowest = -3.40282347e38f;   // a finite start: -inf - -inf is NaN

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

// The sum over columns [c0, c1) of a row, by the whole workgroup; every
// thread gets it.
template <typename T, int Threads>
__device__ __forceinline__ Sum row_sum(const T *z, uint64_t c0, uint64_t c1, float c, Sum *part)
{
    constexpr int N = kVec<T>, U = 4;
    constexpr uint64_t step = (uint64_t)Threads * N;
    Sum a = {kLowest, 0.0f};
    fvec<N> f[U];
    uint64_t at = c0 + (uint64_t)threadIdx.x * N;
    for (; at + (U - 1) * step + N <= c1; at += U * step) {
        vec<T, N> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = *(const GCQ_G vec<T, N> *)(z + at + u * step);
#pragma unroll
        for (int u = 0; u < U; ++u)
            f[u] = to_f32<T, N>(v[u]);
        add_logits<U, N>(a, f, c);
    }
    for (; at < c1; at += step) {
        fvec<N> g[1];
        const int64_t left = (int64_t)(c1 - at);
        g[0] = to_f32<T, N>(load_vec<T, N>(z + at, left));
#pragma unroll
        for (int j = 0; j < N; ++j)
            g[0][j] = j < left ? g[0][j] : -__builtin_inff();
        add_logits<1, N>(a, g, c);
    }
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1)
        a = join(a, Sum{__shfl_xor(a.m, o, kWave), __shfl_xor(a.s, o, kWave)}, c);
    if ((threadIdx.x & (kWave - 1)) == 0)
        part[threadIdx.x / kWave] = a;
    __syncthreads();
    a = part[0];
#pragma unroll
    for (int w = 1; w < Threads / kWave; ++w)
        a = join(a, part[w], c);
    return a;
}

// The sum (or maximum) over the workgroup, in a fixed order; every thread
// gets it.
template <int Threads, bool Max>
__device__ __forceinline__ float block_reduce(float x, float *part)
{
    x = Max ? max_lanes(x) : sum_lanes(x);
    __syncthreads();   // part may still be read
    if ((threadIdx.x & (kWave - 1)) == 0)
        part[threadIdx.x / kWave] = x;
    __syncthreads();
    x = part[0];
#pragma unroll
    for (int w = 1; w < Threads / kWave; ++w)
        x = Max ? fmaxf(x, part[w]) : x + part[w];
    return x;
}

// A row's entries: column (none: 2^32 - 1), probability, and the student's
// logit there.
constexpr uint32_t kNone = 0xFFFFFFFFu;
struct Entries {
    uint32_t col[GCQ_MAX_TOPK];
    float p[GCQ_MAX_TOPK], z[GCQ_MAX_TOPK];
};

template <typename T>
__device__ __forceinline__ float teacher_logit(const Distill &a, uint64_t row, uint32_t j)
{
    if (a.t_f32)
        return ((const GCQ_G float *)a.top)[row * a.top_ld + j];
    return (float)((const GCQ_G T *)a.top)[row * a.top_ld + j];
}

// Fills `e` with the entries in columns [c0, c1); false if the row has none
// of any weight.  `neg_h` (with Loss): sum of p log p.
template <typename T, int Threads, bool Loss>
__device__ __forceinline__ bool load_entries(const Distill &a, uint64_t row, const T *z,
                                             uint64_t c0, uint64_t c1, Entries &e, float *part,
                                             float &neg_h)
{
    float m = -__builtin_inff();
    for (uint32_t j = threadIdx.x; j < a.k; j += Threads) {
        const uint64_t i = row * a.idx_ld + j;
        const uint64_t col = a.idx64 ? (uint64_t)((const GCQ_G int64_t *)a.idx)[i]
                                     : (uint64_t)(int64_t)((const GCQ_G int32_t *)a.idx)[i];
        const bool real = col < a.vocab;
        const float t = real ? teacher_logit<T>(a, row, j) : -__builtin_inff();
        e.col[j] = real ? (uint32_t)col : kNone;
        e.z[j] = col >= c0 && col < c1 ? (float)((const GCQ_G T *)z)[col] : 0.0f;
        e.p[j] = t;
        m = fmaxf(m, t);
    }
    m = block_reduce<Threads, true>(m, part);
    if (m == -__builtin_inff())
        m = 0.0f;   // nothing but absent or -inf entries: the sum is 0 (a NaN shows in it)
    float s = 0.0f;
    for (uint32_t j = threadIdx.x; j < a.k; j += Threads)
        s += expf((e.p[j] - m) / a.temp);
    s = block_reduce<Threads, false>(s, part);
    const float ls = logf(s);
    float h = 0.0f;
    for (uint32_t j = threadIdx.x; j < a.k; j += Threads) {
        const float l = (e.p[j] - m) / a.temp, p = expf(l) / s;
        e.p[j] = p;
        if (p != 0.0f)
            h += p * (l - ls);
    }
    if constexpr (Loss)
        neg_h = block_reduce<Threads, false>(h, part);
    __syncthreads();   // e is whole
    return s != 0.0f;
}

// dz at the entries' columns in [c0, c1), over what the dense pass wrote
// there (after a barrier).  A column named twice loses both probabilities;
// each of its entries writes the same sum.
template <typename T, int Threads, typename Q>
__device__ __forceinline__ void put_entries(const Distill &a, const Entries &e, T *dz, uint64_t c0,
                                            uint64_t c1, float g, Q q)
{
    for (uint32_t j = threadIdx.x; j < a.k; j += Threads) {
        const uint32_t col = e.col[j];
        if (col == kNone || col < c0 || col >= c1)
            continue;
        float p = 0.0f;
        for (uint32_t i = 0; i < a.k; ++i)
            p += e.col[i] == col ? e.p[i] : 0.0f;
        ((GCQ_G T *)dz)[col] = (T)(g * (q(e.z[j]) - p));
    }
}

// dz = value(z) over columns [c0, c1).
template <typename T, int Threads, typename F>
__device__ __forceinline__ void map_row(const T *z, T *dz, uint64_t c0, uint64_t c1, F value)
{
    constexpr int N = kVec<T>, U = 4;
    constexpr uint64_t step = (uint64_t)Threads * N;
    uint64_t at = c0 + (uint64_t)threadIdx.x * N;
    for (; at + (U - 1) * step + N <= c1; at += U * step) {
        vec<T, N> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            v[u] = *(const GCQ_G vec<T, N> *)(z + at + u * step);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            fvec<N> f = to_f32<T, N>(v[u]);
#pragma unroll
            for (int j = 0; j < N; ++j)
                f[j] = value(f[j]);
            *(GCQ_G vec<T, N> *)(dz + at + u * step) = from_f32<T, N>(f);
        }
    }
    for (; at < c1; at += step) {
        const int64_t left = (int64_t)(c1 - at);
        fvec<N> f = to_f32<T, N>(load_vec<T, N>(z + at, left));
#pragma unroll
        for (int j = 0; j < N; ++j)
            f[j] = value(f[j]);
        store_vec<T, N>(dz + at, from_f32<T, N>(f), left);
    }
}

template <typename T, int Threads>
__device__ __forceinline__ void zero_row(T *dz, uint64_t c0, uint64_t c1)
{
    constexpr int N = kVec<T>;
    const vec<T, N> zero = (T)0.0f;
    for (uint64_t at = c0 + (uint64_t)threadIdx.x * N; at < c1; at += (uint64_t)Threads * N)
        store_vec<T, N>(dz + at, zero, (int64_t)(c1 - at));
}

// Loss and lse, and with Grad dz too: a workgroup per row.  The second pass
// finds the row in the caches.
template <typename T, int Threads, bool Grad>
__global__ __launch_bounds__(Threads) void distill_loss_kernel(Distill a)
{
    __shared__ Entries e;
    __shared__ float part[Threads / kWave];
    __shared__ Sum sums[Threads / kWave];
    const uint64_t row = block_number();
    if (row >= a.rows)
        return;
    const T *z = (const T *)a.z + row * a.z_ld;
    T *dz = (T *)a.dz + row * a.dz_ld;
    const float s = a.row_scale ? a.scale * a.row_scale[row] : a.scale;
    if (s == 0.0f) {
        if (threadIdx.x == 0) {
            a.loss[row] = 0.0f;
            a.lse_out[row] = 0.0f;
        }
        if constexpr (Grad)
            zero_row<T, Threads>(dz, 0, a.vocab);
        return;
    }
    float neg_h;
    const bool any = load_entries<T, Threads, true>(a, row, z, 0, a.vocab, e, part, neg_h);
    const float c = kLog2e / a.temp;
    const Sum r = row_sum<T, Threads>(z, 0, a.vocab, c, sums);
    const float lz = logf(r.s);
    float x = 0.0f;   // cross entropy with q
    for (uint32_t j = threadIdx.x; j < a.k; j += Threads)
        if (e.p[j] != 0.0f)
            x += e.p[j] * ((e.z[j] - r.m) / a.temp - lz);
    x = block_reduce<Threads, false>(x, part);
    if (threadIdx.x == 0) {
        // no finite logit: nothing of q is left where p is
        const float kl = r.s == 0.0f ? __builtin_inff() : neg_h - x;
        a.loss[row] = any ? s * kl : 0.0f;
        a.lse_out[row] = r.m / a.temp + lz;
    }
    if constexpr (Grad) {
        if (!any || r.s == 0.0f) {
            zero_row<T, Threads>(dz, 0, a.vocab);
            return;
        }
        const float g = s / a.temp, f = g / r.s, inv = 1.0f / r.s;
        map_row<T, Threads>(z, dz, 0, a.vocab,
                            [=](float v) { return exp2_hw((v - r.m) * c) * f; });
        __syncthreads();
        put_entries<T, Threads>(a, e, dz, 0, a.vocab, g,
                                [=](float v) { return exp2_hw((v - r.m) * c) * inv; });
    }
}

// dz from a kept lse; `parts` workgroups share a row, `chunk` columns each.  The exponent is
// ((z - hi) - lo) log2(e) / T with hi + lo = lse T: exact where q is large.
template <typename T, int Threads>
__global__ __launch_bounds__(Threads) void distill_grad_kernel(Distill a, uint64_t parts,
                                                               uint64_t chunk)
{
    __shared__ Entries e;
    __shared__ float part[Threads / kWave];
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
    float unused;
    if (!load_entries<T, Threads, false>(a, row, z, c0, c1, e, part, unused)) {
        zero_row<T, Threads>(dz, c0, c1);
        return;
    }
    const float c = kLog2e / a.temp, g = s / a.temp;
    const float hi = lse * a.temp, lo = fmaf(lse, a.temp, -hi);
    const auto q = [=](float v) { return exp2_hw(((v - hi) - lo) * c); };
    map_row<T, Threads>(z, dz, c0, c1, [=](float v) { return q(v) * g; });
    __syncthreads();
    put_entries<T, Threads>(a, e, dz, c0, c1, g, q);
}

template <typename T>
hipError_t loss(const Distill &a, hipStream_t s)
{
    const dim3 rows = block_grid(a.rows);
    if (a.dz)
        distill_loss_kernel<T, 512, true><<<rows, 512, 0, s>>>(a);
    else
        distill_loss_kernel<T, 512, false><<<rows, 512, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t grad(const Distill &a, hipStream_t s)
{
    constexpr int threads = 256;
    const uint64_t chunk = (uint64_t)threads * kVec<T> * 16;
    const uint64_t parts = (a.vocab + chunk - 1) / chunk;
    distill_grad_kernel<T, threads>
        <<<block_grid(a.rows * parts), threads, 0, s>>>(a, parts, chunk);
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
