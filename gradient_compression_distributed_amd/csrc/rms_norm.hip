// rms_norm.hip -- root-mean-square norm with the residual's addition, its
// output plain or in 8 bits with scales, and its gradient, for gfx950.
//
//   h = x + residual          (x alone without a residual)
//   rstd = 1 / sqrt(mean(h^2) + eps)
//   y = h * rstd * w
//   8 bits, per group of columns: a = max |y|,
//     scale = 0 if a = 0, else max(a / 448, 2^-126);  code = e4m3(y / scale)
// and for an output gradient dy (the 8-bit rounding passes it straight on)
// and the gradient dh that reaches h by other ways:
//   u = dy * w;  dx = rstd * (u - h * rstd^2 * mean(u * h)) + dh
//   dw = sum over rows of dy * h * rstd
//
// A row stays in the registers of the lanes that share it between the pass
// for its statistics and the pass that uses them, so every matrix is read
// once.  Statistics are taken from h before it is rounded for storing.
#include <algorithm>

#include "gcq_device.h"
#include "gcq_lm.h"

namespace gcq {

namespace {

using namespace lm;

constexpr float kE4m3Max = 448.0f;
constexpr float kMinNormal = 1.17549435e-38f;   // 2^-126: its reciprocal is finite

// Sum (or maximum) over the L lanes of a row; for L > 64 the workgroup is
// one row and `part` holds a value per wavefront.  The caller alternates
// between two parts, so one barrier per reduction is enough.
template <int L, bool Max>
__device__ __forceinline__ float row_reduce(float x, float *part)
{
    x = Max ? max_lanes<L < kWave ? L : kWave>(x) : sum_lanes<L < kWave ? L : kWave>(x);
    if constexpr (L > kWave) {
        if ((threadIdx.x & (kWave - 1)) == 0)
            part[threadIdx.x / kWave] = x;
        __syncthreads();
        x = part[0];
#pragma unroll
        for (int w = 1; w < L / kWave; ++w)
            x = Max ? fmaxf(x, part[w]) : x + part[w];
    }
    return x;
}

template <int N>
__device__ __forceinline__ fvec<N> load_weight(const void *w, bool f32, uint64_t c, int64_t left,
                                               const float *)
{
    return load_vec<float, N>((const float *)w + c, left);
}

template <int N, typename T>
__device__ __forceinline__ fvec<N> load_weight(const void *w, bool f32, uint64_t c, int64_t left,
                                               const T *)
{
    if (f32)
        return load_vec<float, N>((const float *)w + c, left);
    return to_f32<T, N>(load_vec<T, N>((const T *)w + c, left));
}

// Two e4m3 codes per conversion, four per word, lowest byte first.
template <int N>
__device__ __forceinline__ void store_codes(uint8_t *p, fvec<N> v, int64_t left)
{
    uint32_t q[N / 4];
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
        int word = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
        q[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], word, true);
    }
    vec<uint8_t, N> b;
#pragma unroll
    for (int i = 0; i < N; ++i)
        b[i] = (uint8_t)(q[i / 4] >> (8 * (i % 4)));
    store_vec<uint8_t, N>(p, b, left);
}

// How a group's values become codes: its scale and 1 / scale, 0 for a scale of
// 0.
struct Scale {
    float s, inv;
};

// Scale of a group whose largest magnitude is a.
__device__ __forceinline__ Scale group_scale(float a)
{
    const float s = a == 0.0f ? 0.0f : fmaxf(a / kE4m3Max, kMinNormal);
    return {s, s == 0.0f ? 0.0f : 1.0f / s};
}

// y / scale in float32.  The product with the rounded reciprocal misses one tie
// between two codes in eight (129000 of scales 3 .. 2047); its remainder's
// correction (Markstein 1990) makes it the rounded quotient, with two
// operations a value and one division a group.  A scale of infinity leaves
// finite values 0 (their remainder would be NaN).
template <int N>
__device__ __forceinline__ fvec<N> quotient(fvec<N> y, Scale g)
{
    const float s = __builtin_isinf(g.s) ? 0.0f : g.s;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float q = y[j] * g.inv;
        y[j] = fmaf(-fmaf(q, s, -y[j]), g.inv, q);
    }
    return y;
}

// A row's lanes hold Ch vectors of N columns, L * N columns apart.  Nt: x, the
// residual, h and y by non-temporal accesses; the codes are always stored
// ordinarily (non-temporal ones are slower).  Bound by memory: 16384 x 4096
// bf16 with a residual to 8 bits 81 us (472 MB, 5.8 TB/s); few rows take a
// launch (8192 columns on 1024 lanes, 4 us).
template <typename T, int L, int Ch, bool Q8, bool Nt>
__global__ __launch_bounds__(L < 256 ? 256 : L) void rms_norm_kernel(RmsNorm a)
{
    constexpr int N = kVec<T>, Threads = L < 256 ? 256 : L;
    __shared__ float part[2][Threads / kWave];
    const uint32_t lane = threadIdx.x & (L - 1);
    const uint64_t row = block_number() * (Threads / L) + threadIdx.x / L;
    if (row >= a.rows)
        return;   // a whole workgroup, or a wavefront of one without barriers
    const T *x = (const T *)a.x + row * a.x_ld, *res = (const T *)a.res + row * a.res_ld;
    fvec<N> h[Ch];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < Ch; ++i) {
        const uint64_t c = ((uint64_t)i * L + lane) * N;
        h[i] = 0.0f;
        if (c < a.dim) {
            const int64_t left = (int64_t)(a.dim - c);
            h[i] = to_f32<T, N>(load_vec<T, N, Nt>(x + c, left));
            if (a.res)
                h[i] += to_f32<T, N>(load_vec<T, N, Nt>(res + c, left));
            if (a.h)
                store_vec<T, N, Nt>((T *)a.h + row * a.h_ld + c, from_f32<T, N>(h[i]), left);
        }
#pragma unroll
        for (int j = 0; j < N; ++j)
            sum = fmaf(h[i][j], h[i][j], sum);
    }
    sum = row_reduce<L, false>(sum, part[0]);
    const float rstd = 1.0f / sqrtf(sum / (float)a.dim + a.eps);
    if (a.rstd && lane == 0)
        a.rstd[row] = rstd;
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < Ch; ++i) {
        const uint64_t c = ((uint64_t)i * L + lane) * N;
        if (c < a.dim) {
            const int64_t left = (int64_t)(a.dim - c);
            h[i] = h[i] * rstd * load_weight<N>(a.w, a.w_f32, c, left, x);
            if constexpr (!Q8)
                store_vec<T, N, Nt>((T *)a.y + row * a.y_ld + c, from_f32<T, N>(h[i]), left);
        }
        if constexpr (Q8) {
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j)
                m = fmaxf(m, fabsf(h[i][j]));
            top = fmaxf(top, m);
            if (a.group) {   // a group is the columns of group / N neighbouring lanes
                for (uint32_t o = 1; o * N < a.group; o <<= 1)
                    m = fmaxf(m, __shfl_xor(m, (int)o, kWave));
                const Scale g = group_scale(m);
                if (c < a.dim) {
                    if (c % a.group == 0)
                        a.scales[row * a.parts + c / a.group] = g.s;
                    store_codes<N>(a.codes + row * a.y_ld + c, quotient<N>(h[i], g),
                                   (int64_t)(a.dim - c));
                }
            }
        }
    }
    if constexpr (Q8) {
        if (!a.group) {
            const Scale g = group_scale(row_reduce<L, true>(top, part[1]));
            if (lane == 0)
                a.scales[row] = g.s;
#pragma unroll
            for (int i = 0; i < Ch; ++i) {
                const uint64_t c = ((uint64_t)i * L + lane) * N;
                if (c < a.dim)
                    store_codes<N>(a.codes + row * a.y_ld + c, quotient<N>(h[i], g),
                                   (int64_t)(a.dim - c));
            }
        }
    }
}

// Rows too long for the registers of a workgroup: the row is read again for
// each pass (from the caches).  h is written by the last pass, so it may take
// the residual's or x's place.
template <typename T, bool Q8>
__global__ __launch_bounds__(1024) void rms_norm_long_kernel(RmsNorm a)
{
    constexpr int N = kVec<T>, L = 1024;
    __shared__ float part[2][L / kWave];
    const uint64_t row = block_number();
    if (row >= a.rows)
        return;
    const T *x = (const T *)a.x + row * a.x_ld, *res = (const T *)a.res + row * a.res_ld;
    auto load_h = [&](uint64_t c, int64_t left) {
        fvec<N> h = to_f32<T, N>(load_vec<T, N>(x + c, left));
        if (a.res)
            h += to_f32<T, N>(load_vec<T, N>(res + c, left));
        return h;
    };
    const uint64_t step = (uint64_t)L * N, c0 = (uint64_t)threadIdx.x * N;
    float sum = 0.0f;
    for (uint64_t c = c0; c < a.dim; c += step) {
        const fvec<N> h = load_h(c, (int64_t)(a.dim - c));
#pragma unroll
        for (int j = 0; j < N; ++j)
            sum = fmaf(h[j], h[j], sum);
    }
    sum = row_reduce<L, false>(sum, part[0]);
    const float rstd = 1.0f / sqrtf(sum / (float)a.dim + a.eps);
    if (a.rstd && threadIdx.x == 0)
        a.rstd[row] = rstd;
    Scale g = {0.0f, 0.0f};
    if constexpr (Q8) {
        if (!a.group) {
            float top = 0.0f;
            for (uint64_t c = c0; c < a.dim; c += step) {
                const int64_t left = (int64_t)(a.dim - c);
                const fvec<N> y = load_h(c, left) * rstd * load_weight<N>(a.w, a.w_f32, c, left, x);
#pragma unroll
                for (int j = 0; j < N; ++j)
                    top = fmaxf(top, fabsf(y[j]));
            }
            g = group_scale(row_reduce<L, true>(top, part[1]));
            if (threadIdx.x == 0)
                a.scales[row] = g.s;
        }
    }
    // every lane takes part in a group's maximum: whole steps
    for (uint64_t b = 0; b < a.dim; b += step) {
        const uint64_t c = b + c0;
        const int64_t left = (int64_t)a.dim - (int64_t)c;
        fvec<N> y = 0.0f;
        if (left > 0) {
            const fvec<N> h = load_h(c, left);
            y = h * rstd * load_weight<N>(a.w, a.w_f32, c, left, x);
            if (a.h)
                store_vec<T, N>((T *)a.h + row * a.h_ld + c, from_f32<T, N>(h), left);
            if constexpr (!Q8)
                store_vec<T, N>((T *)a.y + row * a.y_ld + c, from_f32<T, N>(y), left);
        }
        if constexpr (Q8) {
            if (a.group) {
                float m = 0.0f;
#pragma unroll
                for (int j = 0; j < N; ++j)
                    m = fmaxf(m, fabsf(y[j]));
                for (uint32_t o = 1; o * N < a.group; o <<= 1)
                    m = fmaxf(m, __shfl_xor(m, (int)o, kWave));
                g = group_scale(m);
                if (left > 0 && c % a.group == 0)
                    a.scales[row * a.parts + c / a.group] = g.s;
            }
            if (left > 0)
                store_codes<N>(a.codes + row * a.y_ld + c, quotient<N>(y, g), left);
        }
    }
}

// ---------------------------------------------------------------- gradient
// L lanes share a row; slot s of them takes rows s, s + slots, ... and keeps its
// share of dw in registers, so dy, h and dh are read once for both gradients.  A
// workgroup adds its slots' shares at the end and writes them to part_w.  The
// weights' sums run in chains: a lane adds its rows' terms in turn, in float32,
// at most rows / slots of them.  Bound by memory: 16384 x 4096 bf16 98 us (537
// MB and 17 MB of shares, 5.7 TB/s), and 5 for the launch that joins the shares.
// Nt: the matrices by non-temporal accesses.
template <typename T, int L, int Ch, bool Nt>
__global__ __launch_bounds__(L < 256 ? 256 : L) void rms_norm_grad_kernel(RmsGrad a)
{
    constexpr int N = kVec<T>, Threads = L < 256 ? 256 : L;
    constexpr uint32_t Per = Threads / L;
    __shared__ float part[2][Threads / kWave];
    const uint32_t lane = threadIdx.x & (L - 1);
    const uint64_t slot = (uint64_t)blockIdx.x * Per + threadIdx.x / L;
    fvec<N> dw[Ch];
#pragma unroll
    for (int i = 0; i < Ch; ++i)
        dw[i] = 0.0f;
    uint32_t turn = 0;
    for (uint64_t row = slot; row < a.rows; row += a.groups * Per, turn ^= 1u) {
        const T *dy = (const T *)a.dy + row * a.dy_ld, *h = (const T *)a.h + row * a.h_ld;
        const T *dh = (const T *)a.dh + row * a.dh_ld;
        vec<T, N> gv[Ch], hv[Ch], dv[Ch];
        const float rstd = a.rstd[row];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < Ch; ++i) {
            const uint64_t c = ((uint64_t)i * L + lane) * N;
            gv[i] = hv[i] = dv[i] = (T)0.0f;
            if (c < a.dim) {
                const int64_t left = (int64_t)(a.dim - c);
                gv[i] = load_vec<T, N, Nt>(dy + c, left);
                hv[i] = load_vec<T, N, Nt>(h + c, left);
                if (a.dh)
                    dv[i] = load_vec<T, N, Nt>(dh + c, left);
            }
        }
#pragma unroll
        for (int i = 0; i < Ch; ++i) {
            const uint64_t c = ((uint64_t)i * L + lane) * N;
            fvec<N> w = 0.0f;
            if (c < a.dim)
                w = load_weight<N>(a.w, a.w_f32, c, (int64_t)(a.dim - c), dy);
            const fvec<N> g = to_f32<T, N>(gv[i]), hf = to_f32<T, N>(hv[i]);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                sum = fmaf(g[j] * w[j], hf[j], sum);
                dw[i][j] = fmaf(g[j], hf[j] * rstd, dw[i][j]);
            }
        }
        sum = row_reduce<L, false>(sum, part[turn]);
        const float k = sum / (float)a.dim * rstd * rstd;
#pragma unroll
        for (int i = 0; i < Ch; ++i) {
            const uint64_t c = ((uint64_t)i * L + lane) * N;
            if (c >= a.dim)
                continue;
            const int64_t left = (int64_t)(a.dim - c);
            const fvec<N> w = load_weight<N>(a.w, a.w_f32, c, left, dy);
            const fvec<N> g = to_f32<T, N>(gv[i]), hf = to_f32<T, N>(hv[i]);
            fvec<N> d = to_f32<T, N>(dv[i]);
#pragma unroll
            for (int j = 0; j < N; ++j)
                d[j] = fmaf(rstd, fmaf(-hf[j], k, g[j] * w[j]), d[j]);
            store_vec<T, N, Nt>((T *)a.dx + row * a.dx_ld + c, from_f32<T, N>(d), left);
        }
    }
    float *pw = a.part_w + (uint64_t)blockIdx.x * a.dim;
    if constexpr (Per == 1) {
#pragma unroll
        for (int i = 0; i < Ch; ++i) {
            const uint64_t c = ((uint64_t)i * L + lane) * N;
            if (c < a.dim)
                store_vec<float, N>(pw + c, dw[i], (int64_t)(a.dim - c));
        }
    } else {
        __shared__ float share[Per][Ch * L * N];
#pragma unroll
        for (int i = 0; i < Ch; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j)
                share[threadIdx.x / L][(i * L + lane) * N + j] = dw[i][j];
        __syncthreads();
        for (uint32_t c = threadIdx.x; c < a.dim; c += Threads) {
            float sum = share[0][c];
#pragma unroll
            for (uint32_t p = 1; p < Per; ++p)
                sum += share[p][c];
            pw[c] = sum;
        }
    }
}

// Long rows: read twice; the workgroup's share of dw lives in its workspace row
// (each element is always the same lane's).
template <typename T>
__global__ __launch_bounds__(1024) void rms_norm_grad_long_kernel(RmsGrad a)
{
    constexpr int N = kVec<T>, L = 1024;
    __shared__ float part[2][L / kWave];
    const uint64_t slot = blockIdx.x, step = (uint64_t)L * N, c0 = (uint64_t)threadIdx.x * N;
    float *pw = a.part_w + slot * a.dim;
    uint32_t turn = 0;
    for (uint64_t row = slot; row < a.rows; row += a.groups, turn ^= 1u) {
        const T *dy = (const T *)a.dy + row * a.dy_ld, *h = (const T *)a.h + row * a.h_ld;
        const T *dh = (const T *)a.dh + row * a.dh_ld;
        const float rstd = a.rstd[row];
        float sum = 0.0f;
        for (uint64_t c = c0; c < a.dim; c += step) {
            const int64_t left = (int64_t)(a.dim - c);
            const fvec<N> g = to_f32<T, N>(load_vec<T, N>(dy + c, left));
            const fvec<N> hf = to_f32<T, N>(load_vec<T, N>(h + c, left));
            const fvec<N> w = load_weight<N>(a.w, a.w_f32, c, left, dy);
#pragma unroll
            for (int j = 0; j < N; ++j)
                sum = fmaf(g[j] * w[j], hf[j], sum);
        }
        sum = row_reduce<L, false>(sum, part[turn]);
        const float k = sum / (float)a.dim * rstd * rstd;
        for (uint64_t c = c0; c < a.dim; c += step) {
            const int64_t left = (int64_t)(a.dim - c);
            const fvec<N> g = to_f32<T, N>(load_vec<T, N>(dy + c, left));
            const fvec<N> hf = to_f32<T, N>(load_vec<T, N>(h + c, left));
            const fvec<N> w = load_weight<N>(a.w, a.w_f32, c, left, dy);
            fvec<N> d = 0.0f, dw = 0.0f;
            if (a.dh)
                d = to_f32<T, N>(load_vec<T, N>(dh + c, left));
            if (row != slot)
                dw = load_vec<float, N>(pw + c, left);
#pragma unroll
            for (int j = 0; j < N; ++j) {
                d[j] = fmaf(rstd, fmaf(-hf[j], k, g[j] * w[j]), d[j]);
                dw[j] = fmaf(g[j], hf[j] * rstd, dw[j]);
            }
            store_vec<T, N>((T *)a.dx + row * a.dx_ld + c, from_f32<T, N>(d), left);
            store_vec<float, N>(pw + c, dw, left);
        }
    }
}

// dw[c] (+)= the shares: 32 columns per workgroup, 32 groups of lanes over every
// 32nd share, their sums in order.  (64 columns and 16 groups leave
// half the compute units idle at 4096 columns; 16 columns use half a line.)
constexpr uint32_t kDwThreads = 1024, kDwCols = 32;
__global__ __launch_bounds__(kDwThreads) void rms_norm_dw_kernel(const float *__restrict__ part_w,
                                                                 uint64_t shares, uint64_t dim,
                                                                 float *__restrict__ dw, bool add)
{
    constexpr uint32_t groups = kDwThreads / kDwCols;
    __shared__ float share[groups][kDwCols];
    const uint32_t lane = threadIdx.x % kDwCols, group = threadIdx.x / kDwCols;
    const uint64_t c = (uint64_t)blockIdx.x * kDwCols + lane;
    float sum = 0.0f;
    if (c < dim) {
#pragma unroll 8
        for (uint64_t s = group; s < shares; s += groups)
            sum += part_w[s * dim + c];
    }
    share[group][lane] = sum;
    __syncthreads();
    if (group == 0 && c < dim) {
        for (uint32_t g = 1; g < groups; ++g)
            sum += share[g][lane];
        dw[c] = add ? dw[c] + sum : sum;
    }
}

// Lanes per row and vectors per lane (0: too long for registers): the fewest
// lanes that take at most `most` vectors each, so few lanes idle.  1024 lanes
// hold 16 float32 or 16 16-bit elements each before they spill.
struct Split {
    int lanes, ch;
};

template <typename T>
Split split_row(uint64_t dim, uint64_t most, bool q8 = false)
{
    const uint64_t vecs = (dim + kVec<T> - 1) / kVec<T>;
    for (int lanes : {16, 64, 256, 512}) {
        const uint64_t ch = (vecs + lanes - 1) / lanes;
        // 16 lanes: two vectors at most (three for 60000 x 384 bf16 35 us, one of
        // 64 lanes 33), and 128 columns at once where a group may be as many
        if (lanes == 16 ? ch <= 2 && ch <= most && (!q8 || kVec<T> == 8)
                        : ch <= most && (lanes < 512 || q8))
            return {lanes, (int)ch};
    }
    const uint64_t ch = (vecs + 1023) / 1024;
    return {1024, ch <= 16 / kVec<T> ? (int)ch : 0};
}

template <typename T, int L, int Ch, bool Q8>
void norm(const RmsNorm &a, hipStream_t s)
{
    constexpr int threads = L < 256 ? 256 : L, per = threads / L;
    // from 32 MiB a matrix the caches no longer hold them until their next use:
    // 8192 x 4096 bf16 47 us against 52, 2048 x 4096 (16 MiB) 14.3 against 14.1
    const auto kernel = a.rows * a.dim * sizeof(T) >= (32ull << 20)
                            ? rms_norm_kernel<T, L, Ch, Q8, true>
                            : rms_norm_kernel<T, L, Ch, Q8, false>;
    kernel<<<block_grid((a.rows + per - 1) / per), threads, 0, s>>>(a);
}

template <typename T, int L, bool Q8>
void norm(const RmsNorm &a, int ch, hipStream_t s)
{
    if (ch == 1)
        norm<T, L, 1, Q8>(a, s);
    else if (ch == 2)
        norm<T, L, 2, Q8>(a, s);
    else if constexpr ((L == 64 || L == 256) && !Q8)
        norm<T, L, 3, Q8>(a, s);
    else if constexpr (L == 1024 && sizeof(T) == 4)
        ch == 3 ? norm<T, L, 3, Q8>(a, s) : norm<T, L, 4, Q8>(a, s);
}

// Short rows share a wavefront: 16 lanes each (60000 x 64 bf16 8.7 us, 64 lanes
// 20).  Many rows get up to three vectors a lane, to 8 bits two and 512 lanes
// before 1024, us: to 8 bits 16000 x 5120 bf16 121 with two of 512 lanes, 153 with
// three of 256; 8192 x 8192 81, one of 1024 lanes 86; plain, 112 and 112, 90
// and 87; 2999 x 2051 float32 plain 10.4 with three of 256 lanes, 14.5 with one
// of 1024; 5500 x 12000 float32 to 8 bits 173 with three of 1024, 211 with four
// of which one is idle.
template <typename T, bool Q8>
void norm(const RmsNorm &a, hipStream_t s)
{
    const Split p = split_row<T>(a.dim, a.rows < 1024 ? 1 : Q8 ? 2 : 3, Q8);
    if (!p.ch)
        rms_norm_long_kernel<T, Q8><<<block_grid(a.rows), 1024, 0, s>>>(a);
    else if (p.lanes == 64)
        norm<T, 64, Q8>(a, p.ch, s);
    else if (p.lanes == 256)
        norm<T, 256, Q8>(a, p.ch, s);
    else if (p.lanes == 1024)
        norm<T, 1024, Q8>(a, p.ch, s);
    else if (p.lanes == 512) {
        if constexpr (Q8)
            norm<T, 512, Q8>(a, p.ch, s);
    } else if constexpr (!Q8 || kVec<T> == 8) {
        norm<T, 16, Q8>(a, p.ch, s);
    }
}

// The gradient's rows: two vectors a lane at most, 16-bit ones three of 256
// lanes before 1024 (16000 x 5120 bf16 127 us against 141; but three of 64
// lanes, 20000 x 1400, 73 against 55; 10000 x 2500 float32 three of 256 78, one
// of 1024 76).
template <typename T>
Split grad_split(uint64_t dim)
{
    const Split p = split_row<T>(dim, 2);
    return p.lanes == 1024 && sizeof(T) == 2 && dim <= 3 * 256 * kVec<T> ? Split{256, 3} : p;
}

// Short rows share a wavefront here, too (60000 x 64 bf16 13 us, 64 lanes each
// 25).  Workgroups of the gradient: what is resident at once, few enough that their
// shares of dw are a small part of the traffic (16384 x 4096 bf16, us for 512 /
// 768 / 1024 / 1536 of 256 lanes: 109 / 101 / 101 / 109; 16000 x 5120, three
// vectors a lane, 768 / 1024: 127 / 156; 1024 lanes, 256 / 512: 8192 x 8192
// bf16 107 / 111, 8192 x 4096 float32 99 / 94).
template <typename T>
uint64_t grad_groups(uint64_t rows, Split p)
{
    const uint64_t most = p.lanes < 256    ? 1024
                          : p.lanes == 256 ? (p.ch == 3 ? 768 : 1024)
                                           : (p.ch * kVec<T> == 4 ? 512 : 256);
    const uint64_t per = p.lanes < 256 ? 256 / p.lanes : 1, all = (rows + per - 1) / per;
    return all < most ? all : most;
}

// The most that any call of up to `rows` rows of up to `dim` columns needs, so
// a workspace for the largest serves every other one: shorter rows have more
// workgroups (16-bit rows of 4096 columns 1024, of 8192 256).  The workgroups
// depend on dim by its split alone, so each split needs the most at the longest
// row that it takes, in vectors: 2 of 16, 64 and 256 lanes, 3 of 256, 1 of 1024.
template <typename T>
uint64_t most_work(uint64_t rows, uint64_t dim)
{
    uint64_t most = dim * grad_groups<T>(rows, grad_split<T>(dim));
    for (uint64_t vecs : {32, 128, 512, 768, 1024}) {
        const uint64_t d = vecs * kVec<T>;
        if (d < dim)
            most = std::max(most, d * grad_groups<T>(rows, grad_split<T>(d)));
    }
    return 4 * most;
}

template <typename T, int L, int Ch>
void norm_grad(const RmsGrad &a, hipStream_t s)
{
    constexpr int threads = L < 256 ? 256 : L;
    const uint32_t grid = (uint32_t)a.groups;
    // from 64 MiB a matrix on: 16384 x 4096 bf16 101 us against 104, but 2048 x
    // 4096 (16 MiB) 26 against 21
    if (a.rows * a.dim * sizeof(T) >= (64ull << 20))
        rms_norm_grad_kernel<T, L, Ch, true><<<grid, threads, 0, s>>>(a);
    else
        rms_norm_grad_kernel<T, L, Ch, false><<<grid, threads, 0, s>>>(a);
}

template <typename T, int L>
void norm_grad(const RmsGrad &a, int ch, hipStream_t s)
{
    if (ch == 1)
        norm_grad<T, L, 1>(a, s);
    else if (ch == 2)
        norm_grad<T, L, 2>(a, s);
    else if constexpr (L == 256 && sizeof(T) == 2)
        norm_grad<T, L, 3>(a, s);
    else if constexpr (L == 1024 && sizeof(T) == 4)
        ch == 3 ? norm_grad<T, L, 3>(a, s) : norm_grad<T, L, 4>(a, s);
}

template <typename T>
hipError_t norm_grad(RmsGrad a, hipStream_t s)
{
    const Split p = grad_split<T>(a.dim);
    a.groups = grad_groups<T>(a.rows, p);
    if (a.rows) {
        if (!p.ch)
            rms_norm_grad_long_kernel<T><<<(uint32_t)a.groups, 1024, 0, s>>>(a);
        else if (p.lanes == 16)
            norm_grad<T, 16>(a, p.ch, s);
        else if (p.lanes == 64)
            norm_grad<T, 64>(a, p.ch, s);
        else if (p.lanes == 256)
            norm_grad<T, 256>(a, p.ch, s);
        else
            norm_grad<T, 1024>(a, p.ch, s);
    }
    rms_norm_dw_kernel<<<(uint32_t)((a.dim + kDwCols - 1) / kDwCols), kDwThreads, 0, s>>>(
        a.part_w, a.groups, a.dim, a.dw, a.add);
    return hipGetLastError();
}

}  // namespace

uint64_t rms_norm_work_bytes(uint64_t rows, uint64_t dim, int type)
{
    return type == GCQ_F32 ? most_work<float>(rows, dim) : most_work<_Float16>(rows, dim);
}

hipError_t launch_rms_norm(const RmsNorm &a, hipStream_t stream)
{
    switch (a.type) {
    case GCQ_F32: a.codes ? norm<float, true>(a, stream) : norm<float, false>(a, stream); break;
    case GCQ_F16: a.codes ? norm<_Float16, true>(a, stream) : norm<_Float16, false>(a, stream); break;
    default: a.codes ? norm<__bf16, true>(a, stream) : norm<__bf16, false>(a, stream); break;
    }
    return hipGetLastError();
}

hipError_t launch_rms_norm_grad(const RmsGrad &a, hipStream_t stream)
{
    switch (a.type) {
    case GCQ_F32: return norm_grad<float>(a, stream);
    case GCQ_F16: return norm_grad<_Float16>(a, stream);
    default: return norm_grad<__bf16>(a, stream);
    }
}

}  // namespace gcq
