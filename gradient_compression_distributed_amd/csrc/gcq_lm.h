// gcq_lm.h -- shared by the language-model operators (embed.hip,
// rms_norm.hip, distill.hip, gcq_api_lm.hip): element types, vector access,
// wavefront reductions and the launchers.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gcq_device.h"
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
// Nt: non-temporal, for what no other workgroup reads.
template <typename T, int N, bool Nt = false>
__device__ __forceinline__ vec<T, N> load_vec(const T *p, int64_t left)
{
    if (left >= N)
        return dev::ld<Nt>((const GCQ_G vec<T, N> *)p);
    vec<T, N> v;
#pragma unroll
    for (int i = 0; i < N; ++i)
        v[i] = i < left ? ((const GCQ_G T *)p)[i] : (T)0.0f;
    return v;
}

template <typename T, int N, bool Nt = false>
__device__ __forceinline__ void store_vec(T *p, vec<T, N> v, int64_t left)
{
    if (left >= N) {
        dev::st<Nt>((GCQ_G vec<T, N> *)p, v);
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

// A launch's workgroups in two dimensions (one dimension holds at most 2^32
// threads), and the workgroup's number among them.
inline dim3 block_grid(uint64_t blocks)
{
    const uint32_t x = blocks < 65536u ? (uint32_t)blocks : 65536u;
    return dim3(x, (uint32_t)((blocks + x - 1) / x));
}

__device__ __forceinline__ uint64_t block_number()
{
    return (uint64_t)blockIdx.y * gridDim.x + blockIdx.x;
}

}  // namespace lm

// ---- embedding ----------------------------------------------------------
// Sorted positions are summed in runs of at most kEmbedRun; a run's open ends
// leave partial sums in the workspace.
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
    uint32_t run;                   // sorted positions per run
    uint32_t *starts;               // workspace: segment starts before each run, in its tile
    uint32_t *tiles;                // workspace: segment starts in each tile, or before it ...
    bool scanned;                   // ... (scanned)
    float *part;                    // workspace: [runs][2][dim] open sums
};

uint64_t embed_plan_words(uint64_t n);
uint64_t embed_work_bytes(uint64_t n, uint64_t dim);
// Fills in the run length and the workspace pointers of `e`.
void embed_work_layout(EmbedGrad &e, void *work);
hipError_t launch_embed_lookup(const EmbedTable &t, const void *tokens, bool tok64, uint64_t n,
                               float scale, void *out, int out_type, uint64_t out_ld,
                               hipStream_t stream);
hipError_t launch_embed_sort(const void *tokens, bool tok64, uint64_t n, uint64_t vocab,
                             uint32_t *plan, hipStream_t stream);
hipError_t launch_embed_grad(const EmbedGrad &e, hipStream_t stream);

// ---- root-mean-square norm ------------------------------------------------
struct RmsNorm {
    int type;
    bool w_f32;                     // w is float32 (else of `type`)
    const void *x, *res, *w;        // res may be null
    uint64_t rows, dim, x_ld, res_ld, y_ld, h_ld;
    float eps;
    void *y;                        // plain output
    uint8_t *codes;                 // or e4m3 codes (rows y_ld apart) and scales
    float *scales;
    uint32_t group;                 // columns per scale; 0: the whole row
    uint64_t parts;                 // scales per row
    void *h;                        // may be null
    float *rstd;                    // may be null
};

struct RmsGrad {
    int type;
    bool w_f32;
    const void *dy, *h, *w, *dh;    // dh may be null
    const float *rstd;
    uint64_t rows, dim, dy_ld, h_ld, dh_ld, dx_ld;
    void *dx;
    float *dw;
    bool add;                       // dw is added to
    float *part_w;                  // workspace: [groups][dim]
    uint64_t groups;                // workgroups
};

uint64_t rms_norm_work_bytes(uint64_t rows, uint64_t dim, int type);
hipError_t launch_rms_norm(const RmsNorm &a, hipStream_t stream);
hipError_t launch_rms_norm_grad(const RmsGrad &a, hipStream_t stream);

// ---- distillation from top logits -----------------------------------------
struct Distill {
    int type;                       // of z, dz and (unless t_f32) the teacher's logits
    bool t_f32, idx64;
    const void *z, *idx, *top;
    uint64_t rows, vocab, z_ld, idx_ld, top_ld, dz_ld;
    uint32_t k;
    float temp, scale;
    const float *row_scale;         // may be null
    const float *lse;               // null: the loss is wanted; else dz from it
    float *loss, *lse_out;
    void *dz;                       // with the loss: may be null
};

hipError_t launch_distill(const Distill &a, hipStream_t stream);

}  // namespace gcq
