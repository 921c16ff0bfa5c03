// gcq_lm.h -- shared by the language-model operators (embed.hip,
// rms_norm.hip, distill.hip, gcq_api_lm.hip): element types, vector access,
// wavefront reductions and the launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gcq_internal.h"

namespace gcq {
namespace lm {

// ---- element types ----------------------------------------------------
// A lane moves 16 bytes per access: 4 float32 or 8 16-bit values.  Rows may
// start at any element, so vectors are aligned to their element only; gfx950
// takes global accesses of any alignment in one instruction (a 16-byte load
// off its alignment costs at most one more cache line).
template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

template <typename T, int N>
using vec = T __attribute__((ext_vector_type(N), aligned(sizeof(T))));

template <int N>
using fvec = float __attribute__((ext_vector_type(N)));

#define GCQ_G __attribute__((address_space(1)))

// v[0..N) = p[0..N), or only the first `left` of them (the rest 0).
template <typename T, int N>
__device__ __forceinline__ vec<T, N> load_vec(const T *p, int64_t left)
{
    if (left >= N)
        return *(const GCQ_G vec<T, N> *)p;
    vec<T, N> v;
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = i < left ? ((const GCQ_G T *)p)[i] : (T)0.0f;
    return v;
}

template <typename T, int N>
__device__ __forceinline__ void store_vec(T *p, vec<T, N> v, int64_t left)
{
    if (left >= N) {
        *(GCQ_G vec<T, N> *)p = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
        if (i < left)
            ((GCQ_G T *)p)[i] = v[i];
}

template <typename T, int N>
__device__ __forceinline__ fvec<N> to_f32(vec<T, N> v)
{
    return __builtin_convertvector(v, fvec<N>);
}

template <typename T, int N>
__device__ __forceinline__ vec<T, N> from_f32(fvec<N> v)
{
    return __builtin_convertvector(v, vec<T, N>);   // to nearest, ties to even
}

// ---- wavefront reductions (every lane gets the result) -----------------
template <int W = kWave>
__device__ __forceinline__ float sum_lanes(float x)
{
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
        x += __shfl_xor(x, o, kWave);
    return x;
}

template <int W = kWave>
__device__ __forceinline__ float max_lanes(float x)
{
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1)
        x = fmaxf(x, __shfl_xor(x, o, kWave));
    return x;
}

}  // namespace lm

// ---- embedding ----------------------------------------------------------
// Sorted positions are summed in runs of kEmbedRun; a run's open ends leave
// partial sums in the workspace.
constexpr uint32_t kEmbedRun = 32;
// Positions per entry of the segment counts.
constexpr uint32_t kEmbedTile = 1024;

struct EmbedTable {
    const void *p;
    int type;
    uint64_t vocab, dim, ld;
};

struct EmbedGrad {
    const void *g;
    int type;
    uint64_t ld;
    const uint32_t *keys, *order;   // sorted tokens, their positions
    uint64_t n, vocab, dim;
    float scale;
    float *out;                     // the dense table's gradient, or the rows
    uint64_t out_ld;
    int32_t *ids, *count;           // row-sparse form (null: dense)
    bool add;                       // dense: add to out; else overwrite
    uint32_t *starts;               // workspace: segment starts before each run, in its tile
    uint32_t *tiles;                // workspace: segment starts before each tile, then all
    float *part;                    // workspace: [runs][2][dim] open sums
};

uint64_t embed_plan_words(uint64_t n);
uint64_t embed_work_bytes(uint64_t n, uint64_t dim);
// Fills in the workspace pointers of `e`.
void embed_work_layout(EmbedGrad &e, void *work);
hipError_t launch_embed_lookup(const EmbedTable &t, const void *tokens, bool tok64, uint64_t n,
                               float scale, void *out, int out_type, uint64_t out_ld,
                               hipStream_t stream);
hipError_t launch_embed_sort(const void *tokens, bool tok64, uint64_t n, uint64_t vocab,
                             uint32_t *plan, hipStream_t stream);
hipError_t launch_embed_grad(const EmbedGrad &e, hipStream_t stream);

}  // namespace gcq
