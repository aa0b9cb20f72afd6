// linear_ce_few.cu -- the products of the linear head's cross entropy for few
// rows of h (a decoding step, a handful of candidates), where reading w once
// is what has to be done:
//   LSE, DZ  z^T = w h^T, the vocabulary along the tiles' rows
//   OUT      dh^T = w^T dz^T, h's columns along the tiles' rows
// The tiles of linear_ce.cu have h's rows along 256 rows of a product and take
// its whole time for one of them (65536 x 768: 17.7 us of products against
// 14.9 us of HBM); here the few rows are the product's short side (16 or 64),
// so that a product takes about as long as its 128 rows of w take to be read
// from shared memory.  The vocabulary is shared out in units of 32 rows, so no
// SM has more than 32 rows more than another.
#include <algorithm>

#include "linear_ce.cuh"
#include "tc.cuh"
#include "tc_pair.cuh"

namespace sn {
namespace ce {
namespace {

constexpr int A_BYTES = 128 * BK * 2;      // 128 rows of w (or 128 columns x 64 rows)
constexpr int EPI_WARPS = 8;               // two for each 32 rows of the tile, half of the columns each
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int SEG = 8, MAX_SEG = 4;        // k blocks of a segment of a logit's sum, segments in tensor memory

template <int NB>
struct Few {
    static constexpr int STAGE = A_BYTES + NB * BK * 2;
    static constexpr int STAGES = NB == 16 ? 11 : 8;
    static constexpr int SMEM = STAGES * STAGE + 1024;
    static constexpr int CW = NB / 2;      // columns of an epilogue warp
};

// CW consecutive fp32 columns of this warp's 32 tensor-memory lanes.
__device__ __forceinline__ void ld_cols(uint32_t a, float (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(a));
    pair::ld_wait(v);
}
__device__ __forceinline__ void ld_cols(uint32_t a, float (&v)[32]) {
    pair::ld32(a, v);
    pair::ld_wait(v);
}

__device__ __forceinline__ void mma_one(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
        : "memory");
}

// One item of a CTA: rows [r0, r1) of the tile's side, k blocks [k0, k1).
struct Item {
    int r0, r1, k0, k1, split;
};
template <int EPI>
__device__ __forceinline__ int item_count(const CeFew& g, int cta, int ctas, int* first) {
    if (EPI == EPI_OUT) {
        const int items = (g.rows + 127) / 128 * g.splits;
        *first = cta;
        return items > cta ? (items - cta - 1) / ctas + 1 : 0;
    }
    const int units = (g.rows + 31) / 32;
    const int u0 = (int)((int64_t)units * cta / ctas), u1 = (int)((int64_t)units * (cta + 1) / ctas);
    *first = u0 * 32;
    return (u1 - u0 + 3) / 4;
}
template <int EPI>
__device__ __forceinline__ Item item_of(const CeFew& g, int i, int first, int cta, int ctas) {
    if (EPI == EPI_OUT) {
        const int tiles = (g.rows + 127) / 128, it = first + i * ctas, split = it / tiles, r0 = (it - split * tiles) * 128;
        return Item{r0, min(g.rows, r0 + 128), (int)((int64_t)g.kblocks * split / g.splits),
                    (int)((int64_t)g.kblocks * (split + 1) / g.splits), split};
    }
    const int units = (g.rows + 31) / 32;
    const int end = (int)((int64_t)units * (cta + 1) / ctas) * 32, r0 = first + i * 128;
    return Item{r0, min(min(g.rows, end), r0 + 128), 0, g.kblocks, 0};
}

template <int EPI, int NB>
__global__ void __launch_bounds__(THREADS, 1)
    ce_few(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap ta128,
           const __grid_constant__ CUtensorMap tb, const CeFew g, SnDevStatus* st, uint64_t limit) {
    using F = Few<NB>;
    constexpr bool AMN = EPI == EPI_OUT;
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t full[F::STAGES], empty[F::STAGES], acc_full[2], acc_empty[2];
    __shared__ uint32_t tslot;
    __shared__ int failed;
    __shared__ int s_target[NB];
    __shared__ float s_lse2[NB], s_gs[NB];
    unsigned char* base = smem_align<1024>(raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x, ctas = gridDim.x;
    int first;
    const int items = item_count<EPI>(g, cta, ctas, &first);
    // logits: segments (see SEG in linear_ce.cu), read out and added whenever there are MAX_SEG of them
    constexpr int seg = EPI == EPI_OUT ? 1 << 30 : SEG, pass = EPI == EPI_OUT ? 1 << 30 : SEG * MAX_SEG;

    if (threadIdx.x == 0) {
        for (int i = 0; i < F::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], EPI_WARPS);
        }
        failed = 0;
        fence_mbar_init();
    }
    if (warp == 1) tc::tmem_alloc(&tslot, 512);
    pdl_trigger();
    pdl_wait();
    const float gmant = EPI == EPI_LSE ? 1.0f : *g.gmant;
    if (EPI != EPI_OUT && threadIdx.x < NB) {
        int target = -1;
        float lse2 = 0.0f, gs = 0.0f;
        if (threadIdx.x < g.N) {
            const int64_t id = load_id(g.targets, g.ids_type, threadIdx.x);
            if (id >= 0 && id < g.V) {
                target = (int)id;
                if (EPI == EPI_DZ) {
                    lse2 = g.lse[threadIdx.x] * LOG2E;
                    gs = g.scale * (g.g != nullptr ? g.g[threadIdx.x] : 1.0f) / gmant;
                }
            }
        }
        s_target[threadIdx.x] = target;
        s_lse2[threadIdx.x] = lse2;
        s_gs[threadIdx.x] = gs;
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = tslot, stage0 = smem_u32(base);

    auto give_up = [&](int site) {
        record_error(st, SN_E_TIMEOUT, (SN_K_LINEAR_CE << 16) | site);
        failed = 1;
    };
    if (warp == 0) {
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            for (int i = 0; i < items && ok; ++i) {
                const Item t = item_of<EPI>(g, i, first, cta, ctas);
                const int boxes = AMN ? 2 : (t.r1 - t.r0 + 31) / 32;
                for (int k = t.k0; k < t.k1; ++k) {
                    if (!mbar_wait(&empty[s], ph ^ 1, limit)) {
                        give_up(5);
                        ok = false;
                        break;
                    }
                    unsigned char* a = base + s * F::STAGE;
                    mbar_arrive_expect_tx(&full[s], boxes * (AMN ? 8192 : 4096) + NB * BK * 2);
                    // (the issuing thread sets the pace: a whole tile's rows are one copy)
                    if (AMN) {
                        tma_load_3d(a, &ta, &full[s], t.r0, k * BK, 0);
                        tma_load_3d(a + 8192, &ta, &full[s], t.r0 + 64, k * BK, 0);
                    } else if (boxes == 4) {
                        tma_load_3d(a, &ta128, &full[s], k * BK, t.r0, 0);
                    } else {
                        for (int j = 0; j < boxes; ++j)
                            tma_load_3d(a + j * 4096, &ta, &full[s], k * BK, t.r0 + 32 * j, 0);
                    }
                    tma_load_3d(a + A_BYTES, &tb, &full[s], k * BK, 0, 0);
                    if (++s == F::STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = pair::idesc_bf16(128, NB, AMN, false);
            int s = 0, turn = 0;   // passes so far
            uint32_t ph = 0;
            bool ok = true;
            for (int i = 0; i < items && ok; ++i) {
                const Item t = item_of<EPI>(g, i, first, cta, ctas);
                for (int p0 = t.k0; p0 < t.k1 && ok; p0 += pass, ++turn) {
                    const int buf = turn & 1, p1 = min(t.k1, p0 + pass);
                    if (!mbar_wait(&acc_empty[buf], ((turn >> 1) & 1) ^ 1, limit)) {
                        give_up(6);
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    for (int k = p0; k < p1; ++k) {
                        if (!mbar_wait(&full[s], ph, limit)) {
                            give_up(7);
                            ok = false;
                            break;
                        }
                        const uint32_t a = stage0 + s * F::STAGE, b = a + A_BYTES;
                        const int kk = k - p0, sg = kk / seg;
                        const uint32_t d = tmem + buf * 256 + sg * NB;
#pragma unroll
                        for (int j = 0; j < BK / 16; ++j)
                            mma_one(d, AMN ? pair::desc_mn_major(a + j * 2048) : pair::desc_k_major(a + j * 32),
                                    pair::desc_k_major(b + j * 32), idesc, kk - sg * seg > 0 || j > 0);
                        tc::commit(&empty[s]);
                        if (++s == F::STAGES) {
                            s = 0;
                            ph ^= 1;
                        }
                    }
                    if (ok) tc::commit(&acc_full[buf]);
                }
            }
        }
    } else {
        const int quad = warp & 3, half = (warp - 2) >> 2;
        constexpr int CW = F::CW;
        const int c0 = half * CW;
        const float c2 = g.scale * LOG2E;
        float mx[CW], sum[CW];
#pragma unroll
        for (int c = 0; c < CW; ++c) {
            mx[c] = -INFINITY;
            sum[c] = 0.0f;
        }
        int turn = 0;
        bool ok = true;
        for (int i = 0; i < items; ++i) {
            const Item t = item_of<EPI>(g, i, first, cta, ctas);
            float v[CW];
            for (int p0 = t.k0; p0 < t.k1; p0 += pass, ++turn) {
                const int buf = turn & 1, segs = (min(t.k1 - p0, pass) - 1) / seg + 1;
                if (!__all_sync(FULL, mbar_wait(&acc_full[buf], (turn >> 1) & 1, limit))) {
                    if (lane == 0) give_up(8);
                    ok = false;
                    break;
                }
                tc::fence_after_sync();
                const uint32_t acc = tmem + buf * 256 + c0 + ((uint32_t)quad << 21);
                const int q0 = p0 == t.k0 ? 1 : 0;
                if (q0 == 1) ld_cols(acc, v);
                for (int q = q0; q < segs; ++q) {
                    float u[CW];
                    ld_cols(acc + q * NB, u);
#pragma unroll
                    for (int c = 0; c < CW; ++c) v[c] += u[c];
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[buf]);
            }
            if (!ok) break;
            const int r = t.r0 + quad * 32 + lane;
            const bool in = r < t.r1;
#pragma unroll
            for (int c = 0; c < CW; ++c) {
                if (c0 + c >= g.N) continue;
                const int col = c0 + c;
                if constexpr (EPI == EPI_LSE) {
                    // each lane keeps the maximum and sum of the vocabulary rows that come to it
                    const float z = in ? v[c] * c2 : -INFINITY, m = fmaxf(mx[c], z);
                    const float ref = m == -INFINITY ? 0.0f : m;
                    sum[c] = sum[c] * ex2(mx[c] - ref) + ex2(z - ref);
                    mx[c] = m;
                    if (in && s_target[col] == r) g.zt[col] = v[c] * g.scale;
                } else if constexpr (EPI == EPI_DZ) {
                    const float p = ex2(fmaf(v[c], c2, -s_lse2[col]));
                    const float d = s_gs[col] * (s_target[col] == g.v0 + r ? p - 1.0f : p);
                    if (in) g.dz[(int64_t)col * g.ldz + r] = from_f32<bf16>(s_target[col] < 0 ? 0.0f : d);
                } else {
                    float* o = g.out + ((int64_t)t.split * g.N + col) * g.ldo + r;
                    if (in) *o = g.add ? *o + v[c] * gmant : v[c] * gmant;
                }
            }
        }
        if constexpr (EPI == EPI_LSE) {
#pragma unroll
            for (int c = 0; c < CW; ++c) {
                if (c0 + c >= g.N) continue;
                float m = mx[c], q = sum[c];
                join_lse_warp(m, q);
                if (lane == 0) g.part[(int64_t)(cta * 4 + quad) * g.N + c0 + c] = make_float2(m, q);
            }
        }
    }
    __syncthreads();
    if (failed) settle();
    __syncthreads();
    if (warp == 1) {
        __syncwarp();
        tc::tmem_dealloc(tmem, 512);
    }
}

template <int EPI, int NB>
cudaError_t run_few(const CUtensorMap& ta, const CUtensorMap& ta128, const CUtensorMap& tb, const CeFew& g, SnDevStatus* st, uint64_t limit,
                    cudaStream_t s) {
    const cudaError_t e = set_smem_attr_once((const void*)ce_few<EPI, NB>, Few<NB>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_after(ce_few<EPI, NB>, SMS, THREADS, Few<NB>::SMEM, 1, s, ta, ta128, tb, g, st, limit);
}

}  // namespace

int few_box(int N) { return N <= 16 ? 16 : FEW_ROWS; }

// As many as give every SM an item, of at least four blocks each, or as a long
// sum needs.
int few_splits(int D, int kblocks) {
    return std::max((int)least_splits(kblocks), std::min(SMS / ((D + 127) / 128), kblocks / 4));
}

cudaError_t launch_few(Epi epi, const CUtensorMap& ta, const CUtensorMap& ta128, const CUtensorMap& tb, const CeFew& g,
                       SnDevStatus* st, uint64_t limit, cudaStream_t s) {
    if (few_box(g.N) == 16)
        return epi == EPI_LSE  ? run_few<EPI_LSE, 16>(ta, ta128, tb, g, st, limit, s)
               : epi == EPI_DZ ? run_few<EPI_DZ, 16>(ta, ta128, tb, g, st, limit, s)
                               : run_few<EPI_OUT, 16>(ta, ta128, tb, g, st, limit, s);
    return epi == EPI_LSE  ? run_few<EPI_LSE, 64>(ta, ta128, tb, g, st, limit, s)
           : epi == EPI_DZ ? run_few<EPI_DZ, 64>(ta, ta128, tb, g, st, limit, s)
                           : run_few<EPI_OUT, 64>(ta, ta128, tb, g, st, limit, s);
}

}  // namespace ce
}  // namespace sn
