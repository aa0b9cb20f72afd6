// linear_ce.cuh -- what the products of the linear head's cross entropy share:
// targets, exponentials and the scale that dz carries.
#pragma once

#include "ptx.cuh"
#include "row_types.cuh"
#include "sn_internal.h"

namespace sn {
namespace ce {

constexpr unsigned FULL = 0xffffffffu;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr int BK = 64;                 // k of one block: 128 bytes of bf16
constexpr int SMS = 152;               // SMs of the GPU this library is for: fixes how sums are cut up
constexpr int MOST_BLOCKS = 256;       // k blocks of a gradient that tensor memory sums at a time (see SEG in linear_ce.cu)
constexpr int64_t least_splits(int64_t kblocks) { return (kblocks + MOST_BLOCKS - 1) / MOST_BLOCKS; }

enum Epi : int { EPI_LSE = 0, EPI_DZ = 1, EPI_OUT = 2 };

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ int64_t load_id(const void* ids, int type, int64_t i) {
    return type == SN_INDEX_I32 ? (int64_t)static_cast<const int32_t*>(ids)[i] : static_cast<const int64_t*>(ids)[i];
}

// dz carries logit_scale * grad_loss without a factor in [1, 2), which the
// products' epilogues put back: that of the first row with a gradient.  Where
// all rows have the same one (a mean over the batch, over its unmasked part)
// and p_t is small, dz_t is then near a power of two and loses next to nothing
// in bf16, instead of the same rounding in every row.  0: x has no such factor.
__device__ __forceinline__ float mantissa(float x) {
    const uint32_t b = __float_as_uint(x), e = (b >> 23) & 0xff;
    return e == 0 || e == 0xff ? 0.0f : __uint_as_float((b & 0x7fffff) | 0x3f800000);
}

// A running maximum (in log2 space) and sum of exponentials, joined with another.
__device__ __forceinline__ void join_lse(float& m, float& sum, float m2, float sum2) {
    const float to = fmaxf(m, m2), ref = to == -INFINITY ? 0.0f : to;
    sum = sum * ex2(m - ref) + sum2 * ex2(m2 - ref);
    m = to;
}
// The same over a warp; every lane ends with the same bits.
__device__ __forceinline__ void join_lse_warp(float& m, float& sum) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float pm = __shfl_xor_sync(FULL, m, o), ps = __shfl_xor_sync(FULL, sum, o);
        // both lanes start from the lower lane's part
        const bool upper = lane & o;
        const float bm = upper ? m : pm, bs = upper ? sum : ps;
        m = upper ? pm : m;
        sum = upper ? ps : sum;
        join_lse(m, sum, bm, bs);
    }
}

// Products with at most FEW_ROWS rows of h (linear_ce_few.cu).
constexpr int FEW_ROWS = 64;
constexpr int FEW_PARTS = 4 * SMS;     // partial maxima and sums of a row
struct CeFew {
    int N;                   // rows of h
    int kblocks;             // ceil(K / 64)
    int rows;                // LSE, DZ: vocabulary rows of this call;  OUT: D
    int v0, V;
    const void* targets;
    int ids_type;
    float scale;
    float2* part;            // LSE: (FEW_PARTS, N)
    float* zt;               // LSE: (N,)
    const float *lse, *g, *gmant;   // DZ, OUT: gmant is the factor that dz leaves out
    bf16* dz;                // DZ: (N, ldz)
    int64_t ldz;
    float* out;              // OUT: (splits, N, ldo) fp32
    int64_t ldo;
    int splits, add;
};
// ta: the vocabulary's rows (LSE, DZ: boxes of 64 k x 32 rows, ta128 the same
// x 128 rows; OUT: of 64 columns x 64 k), tb: boxes of 64 k x few_box(N) rows of
// h or dz.
int few_box(int N);
// Splits of dh's sum over kblocks of the vocabulary.
int few_splits(int D, int kblocks);
cudaError_t launch_few(Epi epi, const CUtensorMap& ta, const CUtensorMap& ta128, const CUtensorMap& tb, const CeFew& g,
                       SnDevStatus* st, uint64_t limit, cudaStream_t s);

}  // namespace ce
}  // namespace sn
