// linear_ce.cu -- softmax cross entropy of a linear head and its gradient,
// without keeping the logits:
//   z = s h w^T,  lse_i = log sum_v exp z_iv,  loss_i = lse_i - z_{i,t_i};
//   dz = s g (exp(z - lse) - onehot(t)),  dh = dz w,  dw = dz^T h.
// All four products run in one kernel, ce_gemm, on the tensor cores; what
// differs is the operands' major order and what becomes of a finished tile:
//   LSE  a tile of z is reduced to each row's maximum and sum of exponentials
//        (in log2 space) over the tile's columns, and the target's logit is
//        picked out; ce_loss joins the tiles of a row;
//   DZ   a tile of z becomes dz, written in bf16 for one piece of the
//        vocabulary;
//   OUT  a tile of dh or dw is stored, or kept in fp32 to be added to (dh over
//        the pieces, either over the splits of a long sum with few tiles).
// fp32 operands are split into three bf16 parts, x = x0 + x1 + x2, and the sum
// runs over the six products of parts that matter at fp32 (x0y0 apart; x0y1,
// x1y0, x1y1, x0y2 and x2y0, 2^-8 of it and less, together; the dropped ones are
// below 2^-24).
#include <algorithm>
#include <climits>
#include <cstring>

#include "linear_ce.cuh"
#include "tc.cuh"
#include "tc_pair.cuh"

namespace sn {
namespace {

using namespace ce;

// A pair of CTAs computes 256 rows x 256 or 512 columns; each has 128 of the
// rows of A, and loads half of the rows of B.
constexpr int BM = 256, BH = 256;
constexpr int BLOCK = 128 * BK * 2;        // 128 rows (or 64 k rows of 128) of one operand: 16 KB
constexpr int EPI_WARPS = 8;               // two for each 32 rows, 128 columns of 256 each
constexpr int HALF = BH / 2;
constexpr int THREADS = 64 + 32 * EPI_WARPS;   // load warp, product warp, epilogue warps
constexpr int OUT_BOX = 4096;              // 32 rows x 128 bytes on their way out, one a warp
constexpr int SMEM = 12 * BLOCK + EPI_WARPS * OUT_BOX + 1024;
constexpr int GROUPS = SMS / 2;

struct CeGemm {
    int M, N;            // tile grid's rows and columns
    int kblocks;         // ceil(K / 64)
    int seg;             // k blocks that are summed in tensor memory at a time (not in wide tiles)
    int bw;              // columns of a tile: 64, 128 or 256, or 512 (wide)
    int mt, nt, splits;  // tiles over rows and columns, splits of the sum
    int items, whole;    // units of work; the first `whole` are whole tiles (wide tiles only)
    // rows of z
    int v0, V;           // vocabulary index of column 0, vocabulary size
    const void* targets;
    int ids_type;
    float scale;
    float2* part;        // LSE: (ceil(N / min(bw, 128)), M) maximum (log2 space) and sum of so many columns
    float* zt;           // LSE: (M,) target logit
    const float *lse, *g, *gmant;   // DZ, OUT: gmant is the factor that dz leaves out
    int planes;          // bf16 parts of the operands, and of dz
    // OUT (and DZ, whose output the tensor map `to` describes): through shared
    // memory and TMA where `tma`, else element by element
    void* out;           // (M, N) of out_f32 ? fp32 : bf16, leading dimension ldo
    int64_t ldo;
    int out_f32, add, tma;
};

// How a pair works on a tile (see ce_gemm).
enum Mode : int { NARROW, WIDE, PARTS };

// bf16 part of (x, y), packed; x and y become what is left (an infinite one
// leaves nothing).
__device__ __forceinline__ uint32_t take_part(float& x, float& y) {
    const uint32_t u = pack_bf16(x, y);
    const float2 f = unpack_bf16(u);
    x = fabsf(f.x) == INFINITY ? 0.0f : x - f.x;
    y = fabsf(f.y) == INFINITY ? 0.0f : y - f.y;
    return u;
}

// Finite values beyond 2^100 (a masked vocabulary row of the type's lowest
// values) count as 2^100: their parts' products have either sign, and must not
// overflow to infinities that cancel to NaN.  Softmax cannot tell them apart.
__device__ __forceinline__ float within_2_100(float x) {
    constexpr float BIG = 1.2676506002282294e30f;
    return fabsf(x) > BIG && fabsf(x) < INFINITY ? copysignf(BIG, x) : x;
}

struct Tile {
    int m, n0, halves, split;   // row tile, first column, 256-column halves (0: nothing to do)
};
// Tiles go in blocks of 16 row tiles, column by column, so that the pairs
// running at one time share few row and column tiles in L2.  Of the wide
// tiles, those from g.whole on, too few for every pair, go as two halves.
template <bool IS_WIDE>
__device__ __forceinline__ Tile tile_of(int item, const CeGemm& g) {
    int only = -1;
    if (IS_WIDE && item >= g.whole) {
        only = (item - g.whole) & 1;
        item = g.whole + ((item - g.whole) >> 1);
    }
    const int tiles = g.mt * g.nt;
    const int split = item / tiles, t = item - split * tiles;
    constexpr int GM = 16;
    const int block = t / (GM * g.nt), first = block * GM;
    const int rows = min(GM, g.mt - first), r = t - block * GM * g.nt;
    Tile x{first + r % rows, (r / rows) * g.bw, 1, split};
    if (IS_WIDE) {
        const int halves = x.n0 + BH < g.N ? 2 : 1;
        x.halves = only < 0 ? halves : only < halves ? 1 : 0;
        if (only > 0) x.n0 += BH;
    }
    return x;
}

// A warp's 32 rows x 128 columns leave through its 4 KB box, 128 bytes a row at
// a time: each lane writes its row's 16-byte pieces at places permuted by the
// row (TMA's 128-byte swizzle, free of bank conflicts), and one TMA store
// writes whole lines, dropping what lies past the tensor's rows and columns.
// Where the rows' pitch is no multiple of 16 bytes, which TMA needs, the warp
// writes the box's rows itself, a line of one row at a time.
struct OutTile {
    const CUtensorMap* map;    // NULL: rows of `out`
    void* out;
    int64_t ldo;
    uint32_t box;
    int n0, row0, plane, rows, ncols, add;   // ncols: columns left from n0
};
__device__ __forceinline__ void box_free(int lane) {
    if (lane == 0) bulk_wait_read_all();
    __syncwarp();
}
// The box is filled: out with it, its first column being c of the tile's.
template <typename Y>
__device__ __forceinline__ void box_out(const OutTile& t, int lane, int c) {
    constexpr int COLS = 128 / sizeof(Y);
    if (t.map != nullptr) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            if (t.add) pair::tma_add(t.map, t.box, t.n0 + c, t.row0, t.plane);
            else pair::tma_store(t.map, t.box, t.n0 + c, t.row0, t.plane);
            bulk_commit();
        }
        return;
    }
    __syncwarp();
    Y* o = static_cast<Y*>(t.out) + (int64_t)t.row0 * t.ldo + t.n0 + c;
    for (int r = 0; r < 32 && t.row0 + r < t.rows; ++r, o += t.ldo) {
#pragma unroll
        for (int j = lane; j < COLS; j += 32) {
            const uint32_t at = t.box + r * 128 + (((j * (int)sizeof(Y) >> 4) ^ (r & 7)) << 4) + (j * (int)sizeof(Y) & 15);
            if (c + j < t.ncols) {
                if constexpr (sizeof(Y) == 4) {
                    uint32_t x;
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
                    reinterpret_cast<uint32_t*>(o)[j] = x;
                } else {
                    uint16_t x;
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at) : "memory");
                    reinterpret_cast<uint16_t*>(o)[j] = x;
                }
            }
        }
    }
    __syncwarp();
}
__device__ __forceinline__ void store_bf16(const OutTile& t, int lane, const float (&v)[HALF]) {
#pragma unroll
    for (int c = 0; c < HALF; c += 64) {
        if (c >= t.ncols) break;
        box_free(lane);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            pair::st_shared_v4(t.box + lane * 128 + ((q ^ (lane & 7)) << 4), pack_bf16(v[c + 8 * q], v[c + 8 * q + 1]),
                               pack_bf16(v[c + 8 * q + 2], v[c + 8 * q + 3]),
                               pack_bf16(v[c + 8 * q + 4], v[c + 8 * q + 5]),
                               pack_bf16(v[c + 8 * q + 6], v[c + 8 * q + 7]));
        box_out<bf16>(t, lane, c);
    }
}
__device__ __forceinline__ void store_f32(const OutTile& t, int lane, const float (&v)[HALF]) {
#pragma unroll
    for (int c = 0; c < HALF; c += 32) {
        if (c >= t.ncols) break;
        box_free(lane);
#pragma unroll
        for (int q = 0; q < 8; ++q)
            pair::st_shared_v4(t.box + lane * 128 + ((q ^ (lane & 7)) << 4), __float_as_uint(v[c + 4 * q]),
                               __float_as_uint(v[c + 4 * q + 1]), __float_as_uint(v[c + 4 * q + 2]),
                               __float_as_uint(v[c + 4 * q + 3]));
        box_out<float>(t, lane, c);
    }
}

// What a warp needs of its rows of a tile, one a lane.
struct Row {
    int row0, row, target;     // first of the warp, this lane's; -1: masked
    float lse2, gs;            // DZ: lse in log2 space; logit_scale * grad_loss without gmant
    bool in;
};

// A finished piece of 32 rows, one a lane, and `width` columns (64 or 128) from n0.
template <int EPI>
__device__ __forceinline__ void finish(const CeGemm& g, const CUtensorMap& to, const Row& r, int n0, int width, int split,
                                       uint32_t box, float gmant, float (&v)[HALF]) {
    const int lane = threadIdx.x & 31, row0 = r.row0, row = r.row, target = r.target;
    const float lse2 = r.lse2, gs = r.gs;
    const bool in = r.in;
    const int ncols = min(width, g.N - n0);
    const int tcol = target - g.v0 - n0;   // the target's column among these, if it is one
    const float c2 = g.scale * LOG2E;
    if constexpr (EPI == EPI_LSE) {
        if (tcol >= 0 && tcol < ncols) {
            float z = 0.0f;
#pragma unroll
            for (int j = 0; j < HALF; ++j) z = tcol == j ? v[j] : z;
            if (target >= 0) g.zt[row] = z * g.scale;
        }
        // the largest logit in log2 space; columns past the vocabulary lose to any
        const float least = c2 < 0.0f ? INFINITY : -INFINITY;
        if (ncols < HALF) {
#pragma unroll
            for (int j = 0; j < HALF; ++j) v[j] = j < ncols ? v[j] : least;
        }
        float m = least;
        if (c2 < 0.0f) {
#pragma unroll
            for (int j = 0; j < HALF; ++j) m = fminf(m, v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < HALF; ++j) m = fmaxf(m, v[j]);
        }
        m = m == least ? -INFINITY : m * c2;
        // all -inf: any finite reference keeps the sum at 0 without inf - inf
        const float ref = m == -INFINITY ? 0.0f : m;
        float sum[4] = {};
        if (ncols < HALF) {
#pragma unroll
            for (int j = 0; j < HALF; ++j) sum[j & 3] += j < ncols ? ex2(fmaf(v[j], c2, -ref)) : 0.0f;
        } else {
#pragma unroll
            for (int j = 0; j < HALF; ++j) sum[j & 3] += ex2(fmaf(v[j], c2, -ref));
        }
        if (in && ncols > 0)
            g.part[(int64_t)(n0 / min(g.bw, HALF)) * g.M + row] =
                make_float2(m, (sum[0] + sum[1]) + (sum[2] + sum[3]));
    } else if constexpr (EPI == EPI_DZ) {
#pragma unroll
        for (int j = 0; j < HALF; ++j) {
            const float p = ex2(fmaf(v[j], c2, -lse2));
            v[j] = gs * p;
        }
        // few warps hold a target's column or a masked row
        if (__any_sync(FULL, tcol >= 0 && tcol < HALF)) {
#pragma unroll
            for (int j = 0; j < HALF; ++j) v[j] = tcol == j ? v[j] - gs : v[j];
        }
        if (__any_sync(FULL, target < 0)) {
#pragma unroll
            for (int j = 0; j < HALF; ++j) v[j] = target < 0 ? 0.0f : v[j];
        }
        if (row0 < g.M && ncols > 0)
            for (int p = 0; p < g.planes; ++p) {
                if (p > 0) {
                    // what the part before has left
#pragma unroll
                    for (int j = 0; j < HALF; ++j) v[j] -= to_f32(from_f32<bf16>(v[j]));
                }
                store_bf16(OutTile{&to, nullptr, 0, box, n0, row0, p, g.M, ncols, 0}, lane, v);
            }
    } else {
#pragma unroll
        for (int j = 0; j < HALF; ++j) v[j] *= gmant;
        if (row0 < g.M && ncols > 0) {
            const OutTile o{g.tma ? &to : nullptr, g.out, g.ldo, box, n0, row0, g.tma ? split : 0, g.M, ncols,
                            g.add};
            if (g.out_f32) store_f32(o, lane, v);
            else store_bf16(o, lane, v);
        }
    }
}

// A pair of CTAs per tile; one thread loads, one of the leader issues products,
// eight warps read finished sums out of tensor memory (512 columns).
// WIDE: tiles of 256 x 512, their two column halves in the two halves of
// tensor memory.  Both halves' products of a k step share A (kept in the
// collector), so that a product reads 3/4 and TMA writes 3/4 of the shared
// memory bytes of a 256 x 256 tile, which those bytes bind: without epilogues,
// 64 of k took a pair 365 ns at 256 x 256, 312 with half of the loads and 309
// with none (4096 x 32000 x 1536).  Half 0 of a tile starts three stages before
// half 1 and ends three before it, so that each half is read out beside
// products of the other.
// NARROW: 256 x 256 (or 128 or 64 where the tiles are few: a block of k then
// takes less time on more pairs), the halves of tensor memory taking turns, which also lets
// a sum be cut into segments of g.seg k blocks that are added in registers.
// PARTS: 256 x 256 of fp32 operands, three bf16 parts each.  A stage holds all
// six blocks of a k block, so that its six products load each part once; the
// large product's sum, cut into segments, has half 0 of tensor memory and the
// five small ones' has half 1.
template <int EPI, bool AMN, bool BMN, Mode MODE>
__global__ void __launch_bounds__(THREADS, 1)
    ce_gemm(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
            const __grid_constant__ CUtensorMap to, const CeGemm g, SnDevStatus* st, uint64_t limit) {
    constexpr bool IS_WIDE = MODE == WIDE;
    constexpr int NA = MODE == PARTS ? 3 : 1, NB = MODE == PARTS ? 3 : MODE == WIDE ? 2 : 1;   // blocks of a stage
    constexpr int STAGE = (NA + NB) * BLOCK, STAGES = 12 / (NA + NB);
    extern __shared__ unsigned char raw[];
    __shared__ uint64_t full[STAGES], empty[STAGES], acc_full[2], acc_empty[2];
    __shared__ uint32_t tslot;
    __shared__ int failed;
    unsigned char* base = smem_align<1024>(raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = pair::cluster_rank();
    const int group = blockIdx.x / 2, groups = gridDim.x / 2;
    const int items = g.items, bw = IS_WIDE ? BH : g.bw;   // columns of one accumulator

    if (threadIdx.x == 0) {
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], 2 * EPI_WARPS);
        }
        failed = 0;
        fence_mbar_init();
    }
    if (warp == 1) pair::tmem_alloc(&tslot, 512);
    tc::fence_before_sync();
    __syncthreads();
    pair::cluster_sync();
    tc::fence_after_sync();
    const uint32_t tmem = tslot;
    const uint32_t stage0 = smem_u32(base);
    pdl_trigger();
    pdl_wait();
    // a wait ran out: the call reports it, every role of the pair comes to its own wait's end
    auto give_up = [&](int site) {
        record_error(st, SN_E_TIMEOUT, (SN_K_LINEAR_CE << 16) | site);
        failed = 1;
    };

    if (warp == 0) {
        if (lane == 0) {
            // loads: each CTA its 128 rows of A and its 128 of every 256 rows of B
            int s = 0;
            uint32_t ph = 0;
            bool ok = true;
            auto load_a = [&](uint32_t dst, uint32_t bar, int m0, int kk, int part) {
                if constexpr (AMN) {
                    for (int j = 0; j < 2; ++j) pair::tma_load(dst + j * 8192, &ta, bar, m0 + 64 * j, kk, part);
                } else {
                    pair::tma_load(dst, &ta, bar, kk, m0, part);
                }
            };
            auto load_b = [&](uint32_t dst, uint32_t bar, int n0, int kk, int part) {
                if constexpr (BMN) {
                    for (int j = 0; j < 2; ++j) pair::tma_load(dst + j * 8192, &tb, bar, n0 + 64 * j, kk, part);
                } else {
                    pair::tma_load(dst, &tb, bar, kk, n0, part);
                }
            };
            for (int item = group; item < items && ok; item += groups) {
                const Tile t = tile_of<IS_WIDE>(item, g);
                if (IS_WIDE && t.halves == 0) continue;
                const int k0 = (int)((int64_t)g.kblocks * t.split / g.splits);
                const int k1 = (int)((int64_t)g.kblocks * (t.split + 1) / g.splits);
                // (of a narrower tile's box of B only the first bw / 2 rows are used)
                const int m0 = t.m * BM + (int)rank * 128, n0 = t.n0 + (int)rank * (bw / 2);
                const int nb = IS_WIDE ? t.halves : NB;
                for (int k = k0; k < k1; ++k) {
                    if (!mbar_wait(&empty[s], ph ^ 1, limit)) {
                        give_up(1);
                        ok = false;
                        break;
                    }
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * (NA + nb) * BLOCK);
                    const uint32_t bar = pair::map_rank(smem_u32(&full[s]), 0), a = stage0 + s * STAGE;
                    for (int q = 0; q < NA; ++q) load_a(a + q * BLOCK, bar, m0, k * BK, q);
                    for (int q = 0; q < nb; ++q)
                        load_b(a + (NA + q) * BLOCK, bar, n0 + (IS_WIDE ? q * BH : 0), k * BK, IS_WIDE ? 0 : q);
                    if (++s == STAGES) {
                        s = 0;
                        ph ^= 1;
                    }
                }
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = pair::idesc_bf16(BM, bw, AMN, BMN);
            const uint64_t da0 = AMN ? pair::desc_mn_major(stage0) : pair::desc_k_major(stage0);
            const uint64_t db0 = BMN ? pair::desc_mn_major(stage0 + NA * BLOCK) : pair::desc_k_major(stage0 + NA * BLOCK);
            // a descriptor's address field counts 16 bytes
            constexpr uint32_t ASTEP = (AMN ? 2048 : 32) / 16, BSTEP = (BMN ? 2048 : 32) / 16;
            constexpr uint32_t QSTEP = BLOCK / 16, SSTEP = STAGE / 16;
            int s = 0;
            uint32_t ph = 0, used[2] = {0, 0};   // uses of each half of tensor memory
            bool ok = true;
            auto take_acc = [&](int b) {
                if (pair::wait_cluster(&acc_empty[b], (used[b] & 1) ^ 1, limit)) {
                    ++used[b];
                    tc::fence_after_sync();
                    return true;
                }
                give_up(2);
                return false;
            };
            auto wait_stage = [&]() {
                if (mbar_wait(&full[s], ph, limit)) return true;
                give_up(3);
                return false;
            };
            auto next_stage = [&]() {
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            };
            // one stage's four products of A block qa and B block qb, A read for them alone
            auto product = [&](int buf, int qa, int qb, bool first) {
#pragma unroll
                for (int j = 0; j < BK / 16; ++j)
                    pair::mma_bf16<pair::A_ONCE>(tmem + buf * BH, da0 + s * SSTEP + qa * QSTEP + j * ASTEP,
                                                 db0 + s * SSTEP + qb * QSTEP + j * BSTEP, idesc, !first || j > 0);
            };
            int turn = 0;
            for (int item = group; item < items && ok; item += groups) {
                const Tile t = tile_of<IS_WIDE>(item, g);
                if (IS_WIDE && t.halves == 0) continue;
                const int k0 = (int)((int64_t)g.kblocks * t.split / g.splits);
                const int k1 = (int)((int64_t)g.kblocks * (t.split + 1) / g.splits);
                if constexpr (MODE == PARTS) {
                    const uint32_t large = tmem, small = tmem + BH;
                    if (!(ok = take_acc(1))) break;
                    for (int k = k0; k < k1; ++k) {
                        if (!(ok = wait_stage())) break;
                        const uint64_t a0 = da0 + s * SSTEP, a1 = a0 + QSTEP, a2 = a1 + QSTEP;
                        const uint64_t b0 = db0 + s * SSTEP, b1 = b0 + QSTEP, b2 = b1 + QSTEP;
                        // the large product stands apart at a segment's start, where its sum may still be read out,
                        // and at the tile's end, where the small ones' is read out beside it
                        const bool starts = (k - k0) % g.seg == 0, last = k == k1 - 1, apart = starts || last;
#pragma unroll
                        for (int j = 0; j < BK / 16; ++j) {
                            const uint32_t ja = j * ASTEP, jb = j * BSTEP;
                            pair::mma_bf16<pair::A_KEEP>(small, a0 + ja, b2 + jb, idesc, k > k0 || j > 0);
                            if (apart) {
                                pair::mma_bf16<pair::A_LAST>(small, a0 + ja, b1 + jb, idesc, true);
                            } else {
                                pair::mma_bf16<pair::A_AGAIN>(small, a0 + ja, b1 + jb, idesc, true);
                                pair::mma_bf16<pair::A_LAST>(large, a0 + ja, b0 + jb, idesc, true);
                            }
                            pair::mma_bf16<pair::A_KEEP>(small, a1 + ja, b1 + jb, idesc, true);
                            pair::mma_bf16<pair::A_LAST>(small, a1 + ja, b0 + jb, idesc, true);
                            pair::mma_bf16<pair::A_ONCE>(small, a2 + ja, b0 + jb, idesc, true);
                        }
                        if (last) pair::commit(&acc_full[1]);
                        if (apart) {
                            if (starts && !(ok = take_acc(0))) break;
                            product(0, 0, 0, starts);
                        }
                        pair::commit(&empty[s]);
                        if (last || (k + 1 - k0) % g.seg == 0) pair::commit(&acc_full[0]);
                        next_stage();
                    }
                } else if (IS_WIDE && t.halves == 2) {
                    // half 0 goes ahead by up to three stages while half 1 is still being read out
                    const int nk = k1 - k0, ahead = min(nk, STAGES - 1), last = min(STAGES - 1, nk - ahead);
                    if (!(ok = take_acc(0))) break;
                    int s0 = s;
                    uint32_t ph0 = ph;
                    for (int k = 0; k < ahead && ok; ++k) {
                        if (!(ok = wait_stage())) break;
                        product(0, 0, 0, k == 0);
                        next_stage();
                    }
                    if (!ok || !(ok = take_acc(1))) break;
                    if (ahead == nk) pair::commit(&acc_full[0]);
                    s = s0;
                    ph = ph0;
                    for (int k = 0; k < ahead; ++k) {
                        product(1, 0, 1, k == 0);
                        pair::commit(&empty[s]);
                        next_stage();
                    }
                    for (int k = ahead; k < nk - last; ++k) {
                        if (!(ok = wait_stage())) break;
                        const uint64_t a = da0 + s * SSTEP, b = db0 + s * SSTEP;
#pragma unroll
                        for (int j = 0; j < BK / 16; ++j) {
                            pair::mma_bf16<pair::A_KEEP>(tmem, a + j * ASTEP, b + j * BSTEP, idesc, true);
                            pair::mma_bf16<pair::A_LAST>(tmem + BH, a + j * ASTEP, b + QSTEP + j * BSTEP, idesc, true);
                        }
                        pair::commit(&empty[s]);
                        next_stage();
                    }
                    if (!ok) break;
                    // the same at the end: half 0 finishes first, and is read out beside half 1's last products
                    if (last > 0) {
                        s0 = s;
                        ph0 = ph;
                        for (int k = 0; k < last && ok; ++k) {
                            if (!(ok = wait_stage())) break;
                            product(0, 0, 0, false);
                            next_stage();
                        }
                        if (!ok) break;
                        pair::commit(&acc_full[0]);
                        s = s0;
                        ph = ph0;
                        for (int k = 0; k < last; ++k) {
                            product(1, 0, 1, false);
                            pair::commit(&empty[s]);
                            next_stage();
                        }
                    }
                    pair::commit(&acc_full[1]);
                } else {
                    const int seg = IS_WIDE ? k1 - k0 : g.seg;
                    for (int ks = k0; ks < k1 && ok; ks += seg) {
                        const int buf = IS_WIDE ? 0 : turn++ & 1, ke = min(k1, ks + seg);
                        if (!(ok = take_acc(buf))) break;
                        for (int k = ks; k < ke; ++k) {
                            if (!(ok = wait_stage())) break;
                            product(buf, 0, 0, k == ks);
                            pair::commit(&empty[s]);
                            next_stage();
                        }
                        if (ok) pair::commit(&acc_full[buf]);
                    }
                }
            }
        }
    } else {
        const int quad = warp & 3, half = (warp - 2) >> 2;
        const float gmant = EPI == EPI_LSE ? 1.0f : *g.gmant;
        const uint32_t box = stage0 + 12 * BLOCK + (warp - 2) * OUT_BOX;
        uint32_t used[2] = {0, 0};
        int turn = 0;
        bool ok = true;
        for (int item = group; item < items && ok; item += groups) {
            const Tile t = tile_of<IS_WIDE>(item, g);
            if (IS_WIDE && t.halves == 0) continue;
            const int k0 = (int)((int64_t)g.kblocks * t.split / g.splits);
            const int k1 = (int)((int64_t)g.kblocks * (t.split + 1) / g.splits);
            // what the rows bring, while the tile is being computed
            Row r{t.m * BM + (int)rank * 128 + quad * 32, 0, -1, 0.0f, 0.0f, false};
            r.row = r.row0 + lane;
            r.in = r.row < g.M;
            if (EPI != EPI_OUT && r.in) {
                const int64_t id = load_id(g.targets, g.ids_type, r.row);
                if (id >= 0 && id < g.V) {
                    r.target = (int)id;
                    if (EPI == EPI_DZ) {
                        r.lse2 = g.lse[r.row] * LOG2E;
                        r.gs = g.scale * (g.g != nullptr ? g.g[r.row] : 1.0f) / gmant;
                    }
                }
            }
            for (int h = 0; h < t.halves && ok; ++h) {
                float v[HALF];
                // this warp's piece of half `buf`, read (first) or added in fp32 to the nearest; the half is free then
                auto gather = [&](int buf, bool first) {
                    if (!__all_sync(FULL, mbar_wait(&acc_full[buf], used[buf] & 1, limit))) {
                        if (lane == 0) give_up(4);
                        return false;
                    }
                    ++used[buf];
                    tc::fence_after_sync();
                    const uint32_t acc = tmem + buf * BH + half * HALF + ((uint32_t)quad << 21);
                    if (first) {
#pragma unroll
                        for (int c = 0; c < HALF; c += 32) pair::ld32(acc + c, v + c);
                        pair::ld_wait(v);
                    } else {
#pragma unroll
                        for (int c = 0; c < HALF; c += 32) {
                            float u[32];
                            pair::ld32(acc + c, u);
                            pair::ld_wait(u);
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[c + j] += u[j];
                        }
                    }
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) pair::arrive_cluster(pair::map_rank(smem_u32(&acc_empty[buf]), 0));
                    return true;
                };
                if constexpr (MODE == WIDE) {
                    ok = gather(h, true);
                } else {
                    for (int ks = k0; ks < k1 && ok; ks += g.seg) {
                        bool first = ks == k0;
                        if (MODE == PARTS && ks + g.seg >= k1) {
                            if (!(ok = gather(1, first))) break;
                            first = false;
                        }
                        ok = gather(MODE == PARTS ? 0 : turn++ & 1, first);
                    }
                }
                if (!ok) break;
                const int width = min(HALF, bw - half * HALF);
                if (width > 0) finish<EPI>(g, to, r, t.n0 + h * BH + half * HALF, width, t.split, box, gmant, v);
            }
        }
        // this thread's stores read their boxes to the end before the CTA goes
        if (lane == 0) bulk_wait_all();
    }
    __syncthreads();
    if (failed) settle();
    pair::cluster_sync();
    if (warp == 1) {
        __syncwarp();
        pair::tmem_free(tmem, 512);
    }
}

// ---------------------------------------------------------------- operands
// Rows of fp32 or bf16 into `planes` bf16 parts of ld columns (ld a multiple
// of 8, zeros past D).  With targets, rows whose target is masked become
// zeros, so that a NaN or infinity in them meets no product (0 x NaN = NaN).
struct Packed {
    int64_t rows;
    const void* x;
    bf16* out;             // (planes, rows, ld)
    const void* targets;
};
// The factor that dz leaves out, in a gradient (see mantissa).
struct Factor {
    float scale;
    const float* g;
    float* out;            // NULL: a forward pass
};
// By one CTA: rows 1024 at a time until one has a gradient.
__device__ void find_factor(const Factor& f, const Packed& h, int ids_type, int V) {
    __shared__ int first;
    if (threadIdx.x == 0) first = INT_MAX;
    __syncthreads();
    float m = f.g == nullptr ? mantissa(f.scale) : 0.0f;
    for (int64_t r0 = 0; f.g != nullptr && r0 < h.rows; r0 += 1024) {
        int mine = INT_MAX;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            const int64_t r = r0 + 256 * i + threadIdx.x;
            if (r >= h.rows) continue;
            const int64_t id = load_id(h.targets, ids_type, r);
            if (mantissa(f.scale * f.g[r]) != 0.0f && id >= 0 && id < V) mine = (int)r;
        }
        if (mine != INT_MAX) atomicMin(&first, mine);
        if (__syncthreads_or(mine != INT_MAX)) {
            m = mantissa(f.scale * f.g[first]);
            break;
        }
    }
    if (threadIdx.x == 0) *f.out = m == 0.0f ? 1.0f : m;
}

// h and w in one launch: the first `first` CTAs have h, the others w (two
// launches cost 2 us more); in a gradient one more has the factor of dz.
template <typename T>
__global__ void __launch_bounds__(256) pack_kernel(Packed h, Packed w, Factor f, int first, int D, int ld, int planes,
                                                   int ids_type, int V) {
    if (f.out != nullptr && blockIdx.x == gridDim.x - 1) {
        pdl_trigger();
        pdl_wait();
        find_factor(f, h, ids_type, V);
        return;
    }
    const bool is_h = (int)blockIdx.x < first;
    const Packed a = is_h ? h : w;
    const T* x = static_cast<const T*>(a.x);
    const int per = ld / 8, cta = is_h ? blockIdx.x : blockIdx.x - first, ctas = is_h ? first : gridDim.x - (f.out != nullptr) - first;
    const int64_t items = a.rows * per, step = (int64_t)ctas * 256, plane = a.rows * ld;
    pdl_trigger();
    pdl_wait();
    const bool vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && D % 8 == 0;
    for (int64_t it = (int64_t)cta * 256 + threadIdx.x; it < items; it += step) {
        const int64_t r = it / per;
        const int c = (int)(it - r * per) * 8;
        bool keep = true;
        if (a.targets != nullptr) {
            const int64_t id = load_id(a.targets, ids_type, r);
            keep = id >= 0 && id < V;
        }
        float v[8] = {};
        if (keep) {
            if (vec) {
                load8(x + r * D + c, v);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float y = to_f32(x[r * D + min(c + i, D - 1)]);
                    v[i] = c + i < D ? y : 0.0f;
                }
            }
        }
        if (planes > 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = within_2_100(v[i]);
        }
        for (int p = 0; p < planes; ++p) {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = planes > 1 ? take_part(v[2 * i], v[2 * i + 1]) : pack_bf16(v[2 * i], v[2 * i + 1]);
            *reinterpret_cast<uint4*>(a.out + p * plane + r * ld + c) = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
}

// ---------------------------------------------------------------- joins
// A row's lse and loss from its tiles' maxima and sums: `rw` rows a CTA (a
// power of two up to 32), whose tiles are shared out among the 32 warps and,
// with fewer than 32 rows, among the lanes.
__global__ void __launch_bounds__(1024) ce_loss(int N, int V, int tiles, int rw, const float2* part, const float* zt,
                                                const void* targets, int ids_type, float* loss, float* lse) {
    __shared__ float2 s[32][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane & (rw - 1), row = blockIdx.x * rw + r, per = 32 / rw;
    pdl_trigger();
    pdl_wait();
    float m = -INFINITY, sum = 0.0f;
    auto join = [&](float2 p) { join_lse(m, sum, p.x, p.y); };
    if (row < N) {
        int t = warp * per + lane / rw;
        for (; t + 3 * 32 * per < tiles; t += 4 * 32 * per) {
            float2 p[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = part[(int64_t)(t + i * 32 * per) * N + row];
#pragma unroll
            for (int i = 0; i < 4; ++i) join(p[i]);
        }
        for (; t < tiles; t += 32 * per) join(part[(int64_t)t * N + row]);
    }
    s[warp][lane] = make_float2(m, sum);
    __syncthreads();
    // warp w joins the 32 x per partial results of row w
    if (warp >= rw) return;
    m = -INFINITY;
    sum = 0.0f;
    for (int i = 0; i < per; ++i) join(s[lane][i * rw + warp]);
    join_lse_warp(m, sum);
    const int out = blockIdx.x * rw + warp;
    if (lane != 0 || out >= N) return;
    const int64_t id = load_id(targets, ids_type, out);
    const bool masked = id < 0 || id >= V;
    const float l = (m + log2f(sum)) * LN2;
    lse[out] = masked ? 0.0f : l;
    if (loss != nullptr) loss[out] = masked ? 0.0f : l - zt[out];
}

// Sum of the n splits' fp32 slices (ld columns a row, a multiple of 8), rounded
// to the output's type.  blockDim = (threads over columns, rows of a CTA).
template <typename Y>
__global__ void __launch_bounds__(256) ce_join(int64_t rows, int D, int64_t ld, const float* slices, int n,
                                               int64_t slice, Y* out) {
    pdl_trigger();
    pdl_wait();
    const bool vec = D % 4 == 0 && (reinterpret_cast<uintptr_t>(out) & (4 * sizeof(Y) - 1)) == 0;
    for (int64_t r = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; r < rows; r += (int64_t)gridDim.x * blockDim.y) {
        for (int c = 4 * threadIdx.x; c < D; c += 4 * blockDim.x) {
            const float* p = slices + r * ld + c;
            float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
            for (int k = 0; k < n; ++k) {
                const float4 x = *reinterpret_cast<const float4*>(p + k * slice);
                s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
            }
            Y* o = out + r * D + c;
            const float v[4] = {s.x, s.y, s.z, s.w};
            if (vec) {
                if constexpr (sizeof(Y) == 4) *reinterpret_cast<float4*>(o) = s;
                else *reinterpret_cast<uint2*>(o) = make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (c + i < D) o[i] = from_f32<Y>(v[i]);
            }
        }
    }
}

// ---------------------------------------------------------------- host
int64_t r256(int64_t x) { return (x + 255) / 256 * 256; }

// k blocks (of 64) summed in tensor memory at a time.  Its fp32 sums are cut,
// not rounded to nearest: each step of 16 loses up to about 2^-24 of the running
// sum, always to the same side (a sum of 512 steps of one sign came out 1.8e-5
// short, of 32 steps 7e-8; dh with a target's large term early in 4096 steps
// 2.4e-4).  fp32 results, and logits in narrow tiles, therefore add
// segments of 32 steps in registers, to the nearest.  Wide tiles have no
// registers for that and take logits of up to 128 steps (D <= 2048; lse is then
// off by 7e-7 of itself, measured).  bf16 gradients, and the five small products
// of fp32 ones, are summed whole, but at most MOST_BLOCKS at a time, longer sums
// in splits that are added in fp32: 1024 steps cut 2^-14 at most, a thirtieth of
// bf16's half step (the gradient of 8000 x 32768 x 1024 takes 980 us with two
// splits of dh, 950 with one).
constexpr int SEG = 8, WHOLE = 32;

// dz of one piece of the vocabulary takes at most this much workspace.
constexpr int64_t PIECE_BYTES = int64_t(512) << 20;

// A split of a long sum has at least so many blocks of k.
int least_blocks(bool f32) { return f32 ? 2 : 8; }

// How a product M x N over kblocks blocks of k is cut up: tiles of 256 rows x bw
// columns, 512 of them (wide), 256, 128 or 64, and the sum in splits whose fp32
// results are added afterwards.  The estimate in us is waves of tiles times a
// tile's time, from measured figures: a block of k takes a pair of CTAs 0.64 us
// wide, 0.37, 0.24 and 0.18 narrower, 2.1, 1.3 and 0.9 with parts, 1.5 more for
// every tile's ends, and slices pass at 6 TB/s.  A last wave of wide tiles that
// fills at most half of the pairs goes as halves.  Narrower tiles or splits win
// where few tiles would leave pairs idle (4096 x 1536 over 500 blocks is 96
// tiles of 256 x 256 for 76 pairs; 116 x 950 is 4).
struct Cut {
    int bw, splits;
    double us;
};
Cut cut_for(int64_t M, int64_t N, int64_t kblocks, bool f32, bool may_wide, bool may_split) {
    Cut best{BH, 1, 1e30};
    const int64_t mt = (M + BM - 1) / BM;
    const int widths[4] = {512, 256, 128, 64};
    const double unit[2][4] = {{0.64, 0.37, 0.24, 0.18}, {0.0, 2.1, 1.3, 0.9}};
    for (int i = may_wide ? 0 : 1; i < 4; ++i) {
        const int64_t nt = (N + widths[i] - 1) / widths[i];
        if (i > 1 && mt * nt > 4 * GROUPS) break;    // many tiles: the wider ones are better
        const int64_t least = may_split ? least_splits(kblocks) : 1;
        for (int64_t s = least; s <= (may_split ? std::max<int64_t>(least, 16) : 1) &&
                                (s == least || kblocks / s >= least_blocks(f32)); ++s) {
            const int64_t tiles = mt * nt * s, tail = tiles % GROUPS;
            const double k = (double)kblocks / s;
            double us = (tiles + GROUPS - 1) / GROUPS * (k * unit[f32][i] + 1.5);
            if (i == 0 && tail > 0 && tail <= GROUPS / 2) us += k * (unit[0][1] - unit[0][0]);
            if (s > 1) us += 4.0 + 8e-6 * M * N * s / 6.0;
            if (us < 0.97 * best.us) best = Cut{widths[i], (int)s, us};
        }
    }
    return best;
}

struct Plan {
    int planes, ld;             // bf16 parts of an operand; columns of packed rows
    bool pack_w, pack_h;
    int vp, pieces;             // vocabulary columns of a piece (the last may have fewer)
    int64_t ldz;
    bool few;                   // at most FEW_ROWS rows: linear_ce_few.cu
    int bw_z;                   // tiles of the logits: forward, or one piece of dz
    Cut h, w;                   // dh over one piece, dw of one piece
    bool dh_slices;
    int64_t o_gmant, o_h, o_w, o_part, o_zt, o_dz, o_dh, o_dw, total;
};

// Partial maxima and sums of a row's logits.
int lse_parts(int V, int bw) { return (V + std::min(bw, HALF) - 1) / std::min(bw, HALF); }

Plan plan_for(int N, int V, int D, int dtype, bool backward) {
    Plan p{};
    const bool f32 = dtype == SN_DTYPE_F32;
    p.planes = f32 ? 3 : 1;
    p.ld = (D + 7) / 8 * 8;
    p.pack_w = f32 || D % 8 != 0;
    p.pack_h = p.pack_w || backward;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        const int64_t o = at;
        at += r256(bytes);
        return o;
    };
    p.o_gmant = backward ? take(4) : 0;
    p.o_h = p.pack_h ? take((int64_t)p.planes * N * p.ld * 2) : 0;
    p.o_w = p.pack_w ? take((int64_t)p.planes * V * p.ld * 2) : 0;
    const int kd = (D + BK - 1) / BK;
    // wide tiles keep a whole sum in tensor memory; up to 256 rows the product
    // is HBM bound and narrow tiles share out w more evenly
    const bool may_wide = !f32 && kd <= WHOLE && N > BM;
    p.bw_z = cut_for(N, V, kd, f32, may_wide, false).bw;
    p.few = !f32 && N <= FEW_ROWS;
    if (!backward) {
        p.o_part = take((int64_t)(p.few ? FEW_PARTS : lse_parts(V, p.bw_z)) * N * 8);
        p.o_zt = take((int64_t)N * 4);
    } else {
        // pieces of the vocabulary: as few as the workspace allows, or a few
        // more where their tiles fill the GPU's waves better
        const int64_t fit = std::max<int64_t>(BH, PIECE_BYTES / ((int64_t)p.planes * N * 2) / BH * BH);
        const int64_t least = (V + fit - 1) / fit;
        double best = 1e30;
        for (int64_t n = least; n <= least + (least > 1 ? 3 : 0); ++n) {
            const int64_t vp = std::min(fit, ((V + n - 1) / n + BH - 1) / BH * BH);
            const int64_t nv = std::min<int64_t>(vp, V);   // columns of the first piece, which fills every slice
            const Cut z = cut_for(N, nv, kd, f32, may_wide, false);
            const Cut h = cut_for(N, D, (nv + BK - 1) / BK, f32, !f32, true);
            const Cut w = cut_for(nv, D, (N + BK - 1) / BK, f32, !f32, true);
            const double us = n * (z.us + h.us + w.us + 10.0 + 8e-6 * N * D / 6.0);
            if (us >= 0.99 * best) continue;
            best = us;
            p.vp = (int)vp;
            p.h = h;
            p.w = w;
        }
        p.pieces = (int)(((int64_t)V + p.vp - 1) / p.vp);
        p.ldz = p.vp;
        p.o_dz = take((int64_t)p.planes * N * p.ldz * 2);
        if (p.few) p.h = Cut{BH, few_splits(D, (std::min(p.vp, V) + BK - 1) / BK), 0.0};
        p.dh_slices = p.few || p.h.splits > 1 || p.pieces > 1;
        p.o_dh = p.dh_slices ? take((int64_t)p.h.splits * N * p.ld * 4) : 0;
        p.o_dw = p.w.splits > 1 ? take((int64_t)p.w.splits * p.vp * p.ld * 4) : 0;
    }
    p.total = at;
    return p;
}

// (planes, rows, cols) of bf16, ld elements a row: boxes of 64 columns x `box` rows.
bool map_bf16(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int planes, int64_t ld, int64_t plane,
              int box) {
    const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)planes};
    const uint64_t str[2] = {(uint64_t)ld * 2, (uint64_t)plane * 2};
    const uint32_t b[3] = {64, (uint32_t)box, 1};
    return encode_tiled_bf16(m, 3, base, dims, str, b);
}
// An epilogue's output: boxes of 128 bytes x 32 rows.
bool map_out(CUtensorMap* m, const void* base, bool f32, int64_t cols, int64_t rows, int planes, int64_t ld,
             int64_t plane) {
    if (!f32) return map_bf16(m, base, cols, rows, planes, ld, plane, 32);
    const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)rows, (uint64_t)planes};
    const uint64_t str[2] = {(uint64_t)ld * 4, (uint64_t)plane * 4};
    const uint32_t b[3] = {32, 32, 1};
    return encode_tiled(m, 3, base, dims, str, b, true);
}

template <int EPI, bool AMN, bool BMN, Mode MODE>
cudaError_t launch_gemm(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& to, CeGemm g,
                        SnDevStatus* st, uint64_t limit, cudaStream_t s) {
    g.mt = (g.M + BM - 1) / BM;
    g.nt = (g.N + g.bw - 1) / g.bw;
    const int64_t tiles = (int64_t)g.mt * g.nt * g.splits, tail = tiles % GROUPS;
    const int64_t halved = MODE == WIDE && tail <= GROUPS / 2 ? tail : 0, items = tiles + halved;
    if (items >= INT32_MAX / 2) return cudaErrorInvalidValue;
    g.whole = (int)(tiles - halved);
    g.items = (int)items;
    cudaError_t e = set_smem_attr_once((const void*)ce_gemm<EPI, AMN, BMN, MODE>, SMEM);
    if (e != cudaSuccess) return e;
    return launch_after(ce_gemm<EPI, AMN, BMN, MODE>, dim3((unsigned)(2 * std::min<int64_t>(items, GROUPS))),
                        dim3(THREADS), SMEM, 2, s, ta, tb, to, g, st, limit);
}

template <int EPI, bool AMN, bool BMN>
cudaError_t run_gemm(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& to, const CeGemm& g,
                     SnDevStatus* st, uint64_t limit, cudaStream_t s) {
    return g.planes > 1 ? launch_gemm<EPI, AMN, BMN, PARTS>(ta, tb, to, g, st, limit, s)
           : g.bw > BH  ? launch_gemm<EPI, AMN, BMN, WIDE>(ta, tb, to, g, st, limit, s)
                        : launch_gemm<EPI, AMN, BMN, NARROW>(ta, tb, to, g, st, limit, s);
}

cudaError_t pack(const Packed& h, const Packed& w, const Factor& f, int D, int ld, int dtype, int planes, int ids_type, int V,
                 cudaStream_t s) {
    auto ctas = [&](const Packed& a) { return (a.rows * (ld / 8) + 255) / 256; };
    const int64_t nh = ctas(h), nw = ctas(w), most = SMS * 8;
    const int64_t first = nh + nw <= most || nw == 0 ? std::min(nh, most)
                                                     : std::max<int64_t>(1, std::min(most - 1, most * nh / (nh + nw)));
    const unsigned grid = (unsigned)std::min(nh + nw, most) + (f.out != nullptr);
    return launch_after(dtype == SN_DTYPE_F32 ? pack_kernel<float> : pack_kernel<bf16>, grid, 256, 0, 1, s, h, w, f, (int)first,
                        D, ld, planes, ids_type, V);
}

cudaError_t join(int64_t rows, int D, int64_t ld, const float* slices, int n, int64_t slice, void* out, int dtype,
                 cudaStream_t s) {
    int tx = 32;
    while (tx < 256 && 4 * tx < D) tx *= 2;
    const int ty = 256 / tx;
    const unsigned grid = (unsigned)std::min<int64_t>((rows + ty - 1) / ty, SMS * 16);
    if (dtype == SN_DTYPE_F32)
        return launch_after(ce_join<float>, grid, dim3(tx, ty), 0, 1, s, rows, D, ld, slices, n, slice, (float*)out);
    return launch_after(ce_join<bf16>, grid, dim3(tx, ty), 0, 1, s, rows, D, ld, slices, n, slice, (bf16*)out);
}

// One gradient product into fp32 slices of the workspace (slices != NULL) or
// straight into the caller's tensor, through TMA where its rows allow it.
template <bool AMN>
cudaError_t gradient(const CUtensorMap& ta, const CUtensorMap& tb, CeGemm g, const Cut& cut, float* slices, int64_t ld,
                     int64_t slice, void* out, bool f32, bool add, SnDevStatus* st, uint64_t limit, cudaStream_t s) {
    CUtensorMap to{};
    if (slices != nullptr) {
        // a last piece may be too short to be split as far; the slices that it
        // leaves alone hold the earlier pieces' sums
        g.splits = std::min<int>(cut.splits, std::max(1, g.kblocks / least_blocks(f32)));
        g.out_f32 = 1;
        g.add = add;
        g.tma = 1;
        if (!map_out(&to, slices, true, g.N, g.M, cut.splits, ld, slice)) return cudaErrorInvalidValue;
    } else {
        g.out = out;
        g.ldo = g.N;
        g.out_f32 = f32;
        g.tma = (int64_t)g.N * (f32 ? 4 : 2) % 16 == 0 && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
        if (g.tma && !map_out(&to, out, f32, g.N, g.M, 1, g.N, (int64_t)g.M * g.N)) return cudaErrorInvalidValue;
    }
    g.bw = cut.bw;
    g.seg = f32 ? SEG : g.kblocks;
    return run_gemm<EPI_OUT, AMN, true>(ta, tb, to, g, st, limit, s);
}

}  // namespace

int64_t linear_ce_ws_bytes(int N, int V, int D, int dtype, bool backward) {
    return plan_for(N, V, D, dtype, backward).total;
}

cudaError_t launch_linear_ce(const LinearCeArgs& x, void* ws, SnDevStatus* st, uint64_t limit, cudaStream_t s) {
    const Plan p = plan_for(x.N, x.V, x.D, x.dtype, x.backward);
    char* w0 = static_cast<char*>(ws);
    cudaError_t e;
    // operands: as they are where TMA can read them, else packed
    const bf16 *h = (const bf16*)x.h, *w = (const bf16*)x.w;
    int64_t hplane = (int64_t)x.N * p.ld, wplane = (int64_t)x.V * p.ld;
    if (p.pack_h) {
        Packed ph{x.N, x.h, (bf16*)(w0 + p.o_h), x.backward ? x.targets : nullptr}, pw{};
        if (p.pack_w) pw = Packed{x.V, x.w, (bf16*)(w0 + p.o_w), nullptr};
        const Factor f{x.logit_scale, x.grad_loss, x.backward ? (float*)(w0 + p.o_gmant) : nullptr};
        e = pack(ph, pw, f, x.D, p.ld, x.dtype, p.planes, x.ids_type, x.V, s);
        if (e != cudaSuccess) return e;
        h = ph.out;
        if (p.pack_w) w = pw.out;
    }
    const int kd = (x.D + BK - 1) / BK;
    const bool f32 = x.dtype == SN_DTYPE_F32;
    CUtensorMap mh, mw, none{};
    if (!map_bf16(&mh, h, p.ld, x.N, p.planes, p.ld, hplane, 128)) return cudaErrorInvalidValue;
    CeGemm g{};
    g.planes = p.planes;
    g.V = x.V;
    g.targets = x.targets;
    g.ids_type = x.ids_type;
    g.scale = x.logit_scale;
    g.splits = 1;
    g.g = x.grad_loss;
    g.gmant = (const float*)(w0 + p.o_gmant);
    CeGemm z = g;       // the logits
    z.M = x.N;
    z.kblocks = kd;
    z.bw = p.bw_z;
    z.seg = p.bw_z > BH ? kd : SEG;
    CeFew few{};
    CUtensorMap mhf, mw32;    // few rows of h; w in boxes of 32 rows
    if (p.few) {
        few.N = x.N;
        few.kblocks = kd;
        few.V = x.V;
        few.targets = x.targets;
        few.ids_type = x.ids_type;
        few.scale = x.logit_scale;
        few.lse = x.lse;
        few.g = x.grad_loss;
        few.gmant = g.gmant;
        if (!map_bf16(&mhf, h, p.ld, x.N, 1, p.ld, hplane, few_box(x.N))) return cudaErrorInvalidValue;
    }
    if (!x.backward) {
        if (!map_bf16(&mw, w, p.ld, x.V, p.planes, p.ld, wplane, 128)) return cudaErrorInvalidValue;
        z.N = x.V;
        z.part = (float2*)(w0 + p.o_part);
        z.zt = (float*)(w0 + p.o_zt);
        if (p.few) {
            few.rows = x.V;
            few.part = z.part;
            few.zt = z.zt;
            if (!map_bf16(&mw32, w, p.ld, x.V, 1, p.ld, wplane, 32)) return cudaErrorInvalidValue;
            e = launch_few(EPI_LSE, mw32, mw, mhf, few, st, limit, s);
        } else {
            e = run_gemm<EPI_LSE, false, false>(mh, mw, none, z, st, limit, s);
        }
        if (e != cudaSuccess) return e;
        const int rw = x.N >= 2048 ? 32 : x.N >= 256 ? 8 : 1;
        return launch_after(ce_loss, (x.N + rw - 1) / rw, 1024, 0, 1, s, x.N, x.V,
                            p.few ? FEW_PARTS : lse_parts(x.V, p.bw_z), rw, z.part, z.zt, x.targets, x.ids_type, x.loss,
                            x.lse_out);
    }
    bf16* dz = (bf16*)(w0 + p.o_dz);
    const int64_t zplane = (int64_t)x.N * p.ldz;
    const int esize = f32 ? 4 : 2;
    CUtensorMap mhn;   // h with K = rows
    if (!map_bf16(&mhn, h, p.ld, x.N, p.planes, p.ld, hplane, BK)) return cudaErrorInvalidValue;
    float* hs = p.dh_slices ? (float*)(w0 + p.o_dh) : nullptr;
    float* wsl = p.w.splits > 1 ? (float*)(w0 + p.o_dw) : nullptr;
    for (int q = 0; q < p.pieces; ++q) {
        const int v0 = q * p.vp, nv = std::min(p.vp, x.V - v0);
        const bf16* wq = w + (int64_t)v0 * p.ld;
        CUtensorMap mwk, mwn, mzk, mzn, mzo;
        if (!map_bf16(&mwk, wq, p.ld, nv, p.planes, p.ld, wplane, 128) ||
            !map_bf16(&mwn, wq, p.ld, nv, p.planes, p.ld, wplane, BK) ||
            !map_bf16(&mzk, dz, nv, x.N, p.planes, p.ldz, zplane, p.few ? few_box(x.N) : 128) ||
            !map_bf16(&mzn, dz, nv, x.N, p.planes, p.ldz, zplane, BK) ||
            !map_out(&mzo, dz, false, nv, x.N, p.planes, p.ldz, zplane))
            return cudaErrorInvalidValue;
        z.N = nv;
        z.v0 = v0;
        z.lse = x.lse;
        if (p.few) {
            few.rows = nv;
            few.v0 = v0;
            few.dz = dz;
            few.ldz = p.ldz;
            if (!map_bf16(&mw32, wq, p.ld, nv, 1, p.ld, wplane, 32)) return cudaErrorInvalidValue;
            e = launch_few(EPI_DZ, mw32, mwk, mhf, few, st, limit, s);
        } else {
            e = run_gemm<EPI_DZ, false, false>(mh, mwk, mzo, z, st, limit, s);
        }
        if (e != cudaSuccess) return e;
        if (x.dh != nullptr && p.few) {
            CeFew f = few;
            f.rows = x.D;
            f.kblocks = (nv + BK - 1) / BK;
            f.out = hs;
            f.ldo = p.ld;
            // a shorter last piece may have fewer splits than slices
            f.splits = std::min(p.h.splits, f.kblocks);
            f.add = q > 0;
            e = launch_few(EPI_OUT, mwn, mwn, mzk, f, st, limit, s);
            if (e != cudaSuccess) return e;
        } else if (x.dh != nullptr) {
            CeGemm b = g;
            b.M = x.N;
            b.N = x.D;
            b.kblocks = (nv + BK - 1) / BK;
            e = gradient<false>(mzk, mwn, b, p.h, hs, p.ld, (int64_t)x.N * p.ld, x.dh, f32, q > 0, st, limit, s);
            if (e != cudaSuccess) return e;
        }
        if (x.dw != nullptr) {
            CeGemm c = g;
            c.M = nv;
            c.N = x.D;
            c.kblocks = (x.N + BK - 1) / BK;
            char* out = static_cast<char*>(x.dw) + (int64_t)v0 * x.D * esize;
            e = gradient<true>(mzn, mhn, c, p.w, wsl, p.ld, (int64_t)p.vp * p.ld, out, f32, false, st, limit, s);
            if (e != cudaSuccess) return e;
            if (wsl != nullptr) {
                e = join(nv, x.D, p.ld, wsl, p.w.splits, (int64_t)p.vp * p.ld, out, x.dtype, s);
                if (e != cudaSuccess) return e;
            }
        }
    }
    if (x.dh != nullptr && hs != nullptr)
        return join(x.N, x.D, p.ld, hs, p.h.splits, (int64_t)x.N * p.ld, x.dh, x.dtype, s);
    return cudaSuccess;
}

}  // namespace sn
