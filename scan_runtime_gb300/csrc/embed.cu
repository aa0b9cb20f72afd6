// embed.cu -- embedding lookup with scaling, out_i = scale * table[ids_i], and
// its gradient, grad_table_v = scale * sum of the grad_out rows of the tokens
// whose id is v.
//
// The gradient sorts the tokens by id (stable), so that a row's tokens are
// neighbours and their sum has one owner and one order; no atomic touches a
// floating-point sum.  Padding tokens (ids outside [0, V)) get the key V and
// sort behind all rows.
#include <algorithm>
#include <climits>

#include "ptx.cuh"
#include "row_types.cuh"
#include "sn_internal.h"

namespace sn {
namespace {

constexpr unsigned FULL = 0xffffffffu;

template <typename I>
__device__ __forceinline__ int token_row(const I* ids, int64_t i, int V) {
    const int64_t id = (int64_t)ids[i];
    return id >= 0 && id < V ? (int)id : -1;
}

// ---------------------------------------------------------------- lookup
template <typename T>
__host__ __device__ constexpr int embed_batch() { return sizeof(T) == 4 ? 1 : 2; }

// A thread copies the same columns of one or two tokens: 8 consecutive ones (VEC,
// 16-byte accesses), else 4 columns blockDim.x apart.  Both types then have 32
// bytes in flight a thread; a CTA does nothing else (16384 x 2048: fp32 36 us
// with one token, 44 with four; bf16 21 with two, 25 with one, 29 with four).
template <typename I, typename T, typename Y, bool VEC>
__global__ void __launch_bounds__(256) embed_kernel(int n, int V, int D, const I* ids, const T* table, float scale,
                                                    Y* out) {
    constexpr int PER = VEC ? 8 : 4, AT_ONCE = embed_batch<T>();
    const int c = blockIdx.y * blockDim.x * PER + threadIdx.x * (VEC ? 8 : 1);
    const int step = gridDim.x * blockDim.y;
    pdl_trigger();
    pdl_wait();
    for (int64_t i0 = blockIdx.x * blockDim.y + threadIdx.y; i0 < n; i0 += (int64_t)step * AT_ONCE) {
        float v[AT_ONCE][PER] = {}, times[AT_ONCE] = {};   // padding's zeros meet no scale (0 x inf = NaN)
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int64_t i = i0 + (int64_t)k * step;
            const int row = i < n ? token_row(ids, i, V) : -1;
            if (row < 0) continue;
            times[k] = scale;
            const T* p = table + (int64_t)row * D;
            if constexpr (VEC) {
                if (c < D) load8(p + c, v[k]);
            } else {
#pragma unroll
                for (int e = 0; e < PER; ++e) v[k][e] = to_f32(p[min(c + e * (int)blockDim.x, D - 1)]);
            }
        }
#pragma unroll
        for (int k = 0; k < AT_ONCE; ++k) {
            const int64_t i = i0 + (int64_t)k * step;
            if (i >= n) break;
            Y* o = out + i * D;
#pragma unroll
            for (int e = 0; e < PER; ++e) v[k][e] *= times[k];
            if constexpr (VEC) {
                if (c < D) store8(o + c, v[k]);
            } else {
#pragma unroll
                for (int e = 0; e < PER; ++e)
                    if (c + e * (int)blockDim.x < D) o[c + e * blockDim.x] = from_f32<Y>(v[k][e]);
            }
        }
    }
}

// ---------------------------------------------------------------- sort by id
// Least-significant-digit radix sort of (key, token) by one cluster of CTAs in
// one launch: the hardware's cluster barrier stands between the passes, where
// a sort over the whole GPU would need three launches a pass.  In each pass a
// warp owns consecutive entries; it counts its digits, the counts of the
// cluster's warps are summed in (digit, CTA, warp) order, and each entry goes
// to its warp's start plus its rank among the warp's equal digits so far, so
// equal keys keep their order.  At most 9 bits a pass: two passes for a
// vocabulary of up to 2^18.
constexpr int SORT_T = 1024, SORT_W = SORT_T / 32, MAX_BINS = 512, MAX_SORT_CTAS = 16;
constexpr int SORT_SMEM = SORT_W * MAX_BINS * 4;

struct SortArgs {
    int n, V, bits, passes;      // bits of a pass's digit
    const void* ids;
    int2* entry[2];              // (key, token); the result is in [passes & 1]
};

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

template <typename I>
__global__ void __launch_bounds__(SORT_T) sort_kernel(SortArgs a) {
    extern __shared__ int at[];            // (SORT_W, MAX_BINS): counts, then next positions
    __shared__ int totals[2][MAX_BINS];    // this CTA's counts, which the cluster's other CTAs read
    __shared__ int wsum[SORT_W];
    constexpr int KEPT = 4;                // a lane's first entries stay in registers between count and placing
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int cta = blockIdx.x, ctas = gridDim.x;
    // entries of this CTA, and of this warp
    const int share = (int)(((int64_t)a.n + ctas * SORT_W - 1) / (ctas * SORT_W));
    const int wshare = (share + 31) / 32 * 32;
    const int64_t lo64 = (int64_t)(cta * SORT_W + warp) * wshare;
    const int lo = (int)min((int64_t)a.n, lo64), hi = (int)min((int64_t)a.n, lo64 + wshare);
    const I* ids = static_cast<const I*>(a.ids);
    int* mine = at + warp * MAX_BINS;
    pdl_trigger();
    pdl_wait();
    for (int p = 0; p < a.passes; ++p) {
        const int shift = p * a.bits, bins = 1 << a.bits;
        const int2* from = a.entry[p & 1];
        int2* to = a.entry[(p + 1) & 1];
        auto load = [&](int i, int& k, int& t) {
            if (p > 0) {
                const int2 e = from[i];
                k = e.x;
                t = e.y;
            } else {
                const int row = token_row(ids, i, a.V);
                k = row >= 0 ? row : a.V;
                t = i;
            }
        };
        int k4[KEPT], t4[KEPT];
#pragma unroll
        for (int c = 0; c < KEPT; ++c)
            if (lo + 32 * c + lane < hi) load(lo + 32 * c + lane, k4[c], t4[c]);
        for (int b = lane; b < bins; b += 32) mine[b] = 0;
        __syncwarp();
#pragma unroll
        for (int c = 0; c < KEPT; ++c)
            if (lo + 32 * c + lane < hi) atomicAdd(&mine[(k4[c] >> shift) & (bins - 1)], 1);
        for (int i = lo + 32 * KEPT + lane; i < hi; i += 32) {
            int k, t;
            load(i, k, t);
            atomicAdd(&mine[(k >> shift) & (bins - 1)], 1);
        }
        __syncthreads();
        // per bin: this CTA's warps' counts, and what of the bin the CTAs before hold
        const int b = threadIdx.x;
        int count[SORT_W], total = 0, before = 0;
        if (b < bins) {
#pragma unroll
            for (int w = 0; w < SORT_W; ++w) count[w] = at[w * MAX_BINS + b];
#pragma unroll
            for (int w = 0; w < SORT_W; ++w) total += count[w];
        }
        if (ctas > 1) {
            if (b < bins) totals[p & 1][b] = total;
            cluster_barrier();
            total = 0;
            if (b < bins) {
                const uint32_t here = smem_u32(&totals[p & 1][b]);
                for (int c0 = 0; c0 < ctas; c0 += 8) {   // 8 or 16 of them
#pragma unroll
                    for (int c = c0; c < c0 + 8; ++c) {
                        uint32_t there;
                        int x;
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(here), "r"(c));
                        asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(x) : "r"(there) : "memory");
                        before += c < cta ? x : 0;
                        total += x;
                    }
                }
            }
        }
        // exclusive sum over the bins, then over the CTA's warps
        int x = total;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(FULL, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) wsum[warp] = x;
        __syncthreads();
        if (b < bins) {
            int start = x - total + before;
            for (int w = 0; w < warp; ++w) start += wsum[w];
#pragma unroll
            for (int w = 0; w < SORT_W; ++w) {
                at[w * MAX_BINS + b] = start;
                start += count[w];
            }
        }
        __syncthreads();
        auto place = [&](bool in, int k, int t) {
            const unsigned act = __ballot_sync(FULL, in);
            if (!in) return;
            const int d = (k >> shift) & (bins - 1);
            const unsigned same = __match_any_sync(act, d);
            const int rank = __popc(same & ((1u << lane) - 1));
            const int dst = mine[d] + rank;
            __syncwarp(act);
            if (rank == 0) mine[d] += __popc(same);
            __syncwarp(act);
            to[dst] = make_int2(k, t);
        };
#pragma unroll
        for (int c = 0; c < KEPT; ++c)
            if (lo + 32 * c < hi) place(lo + 32 * c + lane < hi, k4[c], t4[c]);
        for (int base = lo + 32 * KEPT; base < hi; base += 32) {
            const bool in = base + lane < hi;
            int k = 0, t = 0;
            if (in) load(base + lane, k, t);
            place(in, k, t);
        }
        // the next pass reads what the other warps and CTAs have placed (and no
        // CTA ends while another reads its totals)
        if (ctas > 1) cluster_barrier();
        else __syncthreads();
    }
}

// ---------------------------------------------------------------- sums
// The sorted tokens and the ends of the V rows, merged (a row's tokens, then
// its end), make n + V items: a token costs the read of a gradient row, an end
// the write of a table row.  Every unit takes the same number of consecutive
// items, so that neither a token that fills a tenth of the batch nor a stretch
// of rows without tokens makes a unit longer than the others.  A row whose
// tokens cross units is summed from its units' parts, in order: each unit
// before the last leaves a tail, the last one a head, and join_rows adds them.
struct SumArgs {
    int n, V, D, ipu, units, accumulate;   // ipu: items of a unit
    const int2* entry;        // (key, token), sorted
    const void* g;
    float scale;
    void* out;
    float *tail, *head;       // (slots, D)
    int by_token;             // slots are numbered by token (fewer tokens than units), else by unit
    int* head_row;            // (units,) row whose head the unit holds, or -1
    int *tail_row, *tail_slot;   // (units,) row whose tail the unit holds, or -1, and where it is
};

// Row ends among the first d merged items, by half a warp: the smallest i in
// [max(0, d - n), min(d, V)] for which the i-th row end does not come before
// token d - 1 - i; a round narrows the range to a sixteenth.
__device__ __forceinline__ int ends_before(const int2* entry, int n, int V, int64_t d) {
    const int lane = threadIdx.x & 15;
    const unsigned shift = threadIdx.x & 16;
    int64_t lo = d > n ? d - n : 0, hi = d < V ? d : V;
    while (__any_sync(FULL, lo < hi)) {
        const int64_t len = hi - lo, mid = lo + len * lane / 16;
        const bool before = len > 0 && mid < entry[d - 1 - mid].x;
        const int c = __popc((__ballot_sync(FULL, before) >> shift) & 0xffff);   // true for the first c lanes
        if (len > 0) {
            const int64_t to = c < 16 ? lo + len * c / 16 : hi;
            if (c > 0) lo = lo + len * (c - 1) / 16 + 1;
            hi = to;
        }
    }
    return (int)lo;
}

// A thread holds 8 columns: consecutive ones (VEC, 16-byte accesses), else
// columns blockDim.x apart.  get: zeros past the row's end.
template <bool VEC, typename T>
__device__ __forceinline__ void get_cols(const T* p, int c, int D, float (&v)[8]) {
    if constexpr (VEC) {
        if (c < D) load8(p + c, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            // a load that no branch guards is one of eight in flight
            const int at = c + i * (int)blockDim.x;
            const float x = to_f32(p[min(at, D - 1)]);
            v[i] = at < D ? x : 0.0f;
        }
    }
}
template <bool VEC, typename Y>
__device__ __forceinline__ void put_cols(Y* p, int c, int D, const float (&s)[8]) {
    if constexpr (VEC) {
        if (c < D) store8(p + c, s);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i * (int)blockDim.x < D) p[c + i * blockDim.x] = from_f32<Y>(s[i]);
    }
}

constexpr int MAX_IPU = 64, SUM_T = 256, BATCH = 4;   // tokens whose rows are loaded at a time

// blockDim = (threads over columns, units of a CTA); blockIdx.y: slab of 8 blockDim.x columns.
template <typename T, typename Y, bool VEC>
__global__ void __launch_bounds__(SUM_T, VEC ? 4 : 2) row_sums(SumArgs a) {
    __shared__ int s_key[SUM_T / 32][MAX_IPU + 1], s_tok[SUM_T / 32][MAX_IPU], s_edge[SUM_T / 32][2];
    __shared__ __align__(16) Y zeros[VEC ? 8 * SUM_T : 8];
    const int u = blockIdx.x * blockDim.y + threadIdx.y, ty = threadIdx.y;
    const int64_t d0 = (int64_t)u * a.ipu, d1 = min(d0 + a.ipu, (int64_t)a.n + a.V);
    const bool live = u < a.units;
    if constexpr (VEC)
        for (int k = threadIdx.y * blockDim.x + threadIdx.x; k < (int)sizeof(zeros) / 16; k += blockDim.x * blockDim.y)
            reinterpret_cast<uint4*>(zeros)[k] = make_uint4(0, 0, 0, 0);
    pdl_trigger();
    pdl_wait();
    if (live && threadIdx.x < 32) {
        const int e = ends_before(a.entry, a.n, a.V, threadIdx.x < 16 ? d0 : d1);
        if ((threadIdx.x & 15) == 0) s_edge[ty][threadIdx.x >> 4] = e;
    }
    __syncthreads();
    const int i0 = live ? s_edge[ty][0] : 0, i1 = live ? s_edge[ty][1] : 0;
    const int j0 = live ? (int)(d0 - i0) : 0, j1 = live ? (int)(d1 - i1) : 0;
    for (int k = threadIdx.x; k <= j1 - j0; k += blockDim.x) {
        const int2 e = k < j1 - j0 ? a.entry[j0 + k] : make_int2(INT_MAX, 0);
        s_key[ty][k] = e.x;
        if (k < j1 - j0) s_tok[ty][k] = e.y;
    }
    if constexpr (VEC) fence_proxy_async_smem();
    __syncthreads();
    if (!live) return;
    const int D = a.D, c = blockIdx.y * blockDim.x * 8 + threadIdx.x * (VEC ? 8 : 1);
    const int* key = s_key[ty];
    const bool open = i0 < a.V && j0 > 0 && a.entry[j0 - 1].x == i0;   // row i0 has tokens in the unit before
    const T* g = static_cast<const T*>(a.g);
    Y* out = static_cast<Y*>(a.out);
    // padding tokens (key V) lie behind all rows
    int nt = j1 - j0;
    while (nt > 0 && key[nt - 1] >= a.V) --nt;

    // rows without tokens: zeros, written by the copy engine, a row at a time;
    // one thread issues all of them, in fp32 one of each warp its share (16384
    // tokens, 65536 x 2048: fp32 133.5 against 138 us, bf16 95 against 92)
    constexpr bool SHARED_OUT = sizeof(Y) == 4;
    const bool issuer = SHARED_OUT ? (threadIdx.x & 31) == 0 : threadIdx.x == 0;
    if (!a.accumulate) {
        int j = 0;
        unsigned turn = 0;
        for (int i = i0; i < i1; ++i) {
            const int from = j;
            while (j < nt && key[j] == i) ++j;
            if (j > from || (i == i0 && open)) continue;
            if constexpr (VEC) {
                const int c0 = blockIdx.y * blockDim.x * 8;
                if (threadIdx.x == turn)
                    bulk_store(out + (int64_t)i * D + c0, zeros, min(D - c0, (int)blockDim.x * 8) * (int)sizeof(Y));
                if (SHARED_OUT) turn = turn + 32 < blockDim.x ? turn + 32 : 0;
            } else {
                const float z[8] = {};
                put_cols<VEC>(out + (int64_t)i * D, c, D, z);
            }
        }
        if (VEC && issuer) bulk_commit();
    }

    // a row that ends here without a token of this unit has an empty head
    float s[8] = {};
    if (open && i1 > i0 && (nt == 0 || key[0] != i0))
        put_cols<VEC>(a.head + (a.by_token ? j0 - 1 : u) * (int64_t)D, c, D, s);
    int tail_slot = -1;
    int from = 0;
    for (int t0 = 0; t0 < nt; t0 += BATCH) {
        float v[BATCH][8] = {};
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
            if (t0 + b < nt) get_cols<VEC>(g + (int64_t)s_tok[ty][t0 + b] * D, c, D, v[b]);
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int t = t0 + b;
            if (t >= nt) break;
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] += v[b][k];
            const int i = key[t];
            if (t + 1 < nt && key[t + 1] == i) continue;
            if (i == i1) {
                // the row goes on in the next unit
                tail_slot = a.by_token ? j0 + from : u;
                put_cols<VEC>(a.tail + (int64_t)tail_slot * D, c, D, s);
            } else if (i == i0 && open) {
                // beside the tail of the unit before, whose slot ends at token j0 - 1
                put_cols<VEC>(a.head + (a.by_token ? j0 - 1 : u) * (int64_t)D, c, D, s);
            } else {
                Y* o = out + (int64_t)i * D;
                float old[8] = {};
                if (a.accumulate) get_cols<VEC>(o, c, D, old);
#pragma unroll
                for (int k = 0; k < 8; ++k) s[k] = fmaf(s[k], a.scale, old[k]);
                put_cols<VEC>(o, c, D, s);
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) s[k] = 0.0f;
            from = t + 1;
        }
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) {
        a.head_row[u] = open && i1 > i0 ? i0 : -1;
        a.tail_row[u] = tail_slot >= 0 ? i1 : -1;
        a.tail_slot[u] = tail_slot;
    }
    // the zeros' source is this CTA's
    if (VEC && issuer && !a.accumulate) bulk_wait_all();
}

// Rows that cross units: the tails of the units where the row's tokens are,
// then the head, in that order.  A warp takes 128 columns of the heads of a few
// units; up to 16 tails are in flight at a time.
// BY_UNITS, for at least four tokens a row: rows may then have hundreds of tails
// (a small vocabulary, the frequent ids of a skewed one).  The warps of a CTA
// have different units and the same columns, and add an eighth each of a row
// with many tails, so that its columns are shared out among the SMs (262144
// tokens, 259 x 512: 131 -> 109 us).  With fewer tokens they have the same
// units, whose bookkeeping they then share (16384 tokens, 65536 x 2048 bf16: 92
// against 98 us).
constexpr int JOIN_COLS = 128, JOIN_T = 256, JOIN_W = JOIN_T / 32, LONG_ROW = 96;

template <typename Y, bool BY_UNITS>
__global__ void __launch_bounds__(JOIN_T) join_rows(SumArgs a, int per_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = a.D;
    const int slabs = (D + JOIN_COLS - 1) / JOIN_COLS, groups = (a.units + per_warp - 1) / per_warp;
    const int64_t w0 = (int64_t)blockIdx.x * JOIN_W;
    const bool vec = D % 4 == 0;
    auto col_of = [&](int w) { return (int)(BY_UNITS ? (w0 + w) / groups : (w0 + w) % slabs) * JOIN_COLS + 4 * lane; };
    pdl_trigger();
    pdl_wait();
    auto get = [&](const float* p, int c) {
        const int wide = D - c;     // columns from this lane's first on
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (vec) {
            if (wide > 0) x = *reinterpret_cast<const float4*>(p + c);
        } else {
            if (wide > 0) x.x = p[c];
            if (wide > 1) x.y = p[c + 1];
            if (wide > 2) x.z = p[c + 2];
            if (wide > 3) x.w = p[c + 3];
        }
        return x;
    };
    // sum of the tails of units [from, to)
    auto tails = [&](int from, int to, int c) {
        float4 t = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int f0 = from; f0 < to; f0 += 16) {
            float4 x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (f0 + i < to) x[i] = get(a.tail + (int64_t)(a.by_token ? a.tail_slot[f0 + i] : f0 + i) * D, c);
#pragma unroll
            for (int i = 0; i < 16; ++i)
                if (f0 + i < to) {
                    t.x += x[i].x; t.y += x[i].y; t.z += x[i].z; t.w += x[i].w;
                }
        }
        return t;
    };
    auto finish = [&](int u, int row, int c, const float4& t) {
        const float4 last = get(a.head + (a.by_token ? (int64_t)u * a.ipu - row - 1 : u) * D, c);
        const float v[4] = {t.x + last.x, t.y + last.y, t.z + last.z, t.w + last.w};
        Y* out = static_cast<Y*>(a.out) + (int64_t)row * D + c;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (c + i < D) out[i] = from_f32<Y>(fmaf(v[i], a.scale, a.accumulate ? to_f32(out[i]) : 0.0f));
    };
    const int u0 = (int)(BY_UNITS ? (w0 + warp) % groups : (w0 + warp) / slabs) * per_warp, c = col_of(warp);
    int long_u = 0, long_m = 0, long_row = 0;
    for (int u = u0; u < min(a.units, u0 + per_warp) && c - 4 * lane < D; ++u) {
        const int row = a.head_row[u];
        if (row < 0) continue;
        // the units before with a tail of this row, one run of them: 32 are
        // looked at a time, in strides that grow while all of them are its
        int m = 0;
        for (int stride = 1;;) {
            const int f = u - 1 - m - stride * lane;
            const unsigned same = __ballot_sync(FULL, f >= 0 && a.tail_row[f] == row);
            const int k = same == FULL ? 32 : __ffs(~same) - 1;
            if (k > 0) m += stride * (k - 1) + 1;
            if (k == 32) stride *= 32;
            else if (stride > 1) stride /= 32;
            else break;
        }
        if (BY_UNITS && m >= LONG_ROW && long_m == 0) {
            long_u = u;
            long_m = m;
            long_row = row;
            continue;
        }
        finish(u, row, c, tails(u - m, u, c));
    }
    if constexpr (!BY_UNITS) return;
    __shared__ int s_u[JOIN_W], s_m[JOIN_W];   // a long row of each warp: unit of its head, number of tails
    __shared__ float4 s_sum[JOIN_W][JOIN_W][32];
    if (lane == 0) {
        s_u[warp] = long_u;
        s_m[warp] = long_m;
    }
    if (__syncthreads_or(long_m) == 0) return;
    for (int w = 0; w < JOIN_W; ++w) {
        const int64_t m = s_m[w];
        const int from = s_u[w] - (int)m;
        if (m > 0)
            s_sum[w][warp][lane] = tails(from + (int)(m * warp / JOIN_W), from + (int)(m * (warp + 1) / JOIN_W), col_of(w));
    }
    __syncthreads();
    if (long_m == 0) return;
    float4 t = s_sum[warp][0][lane];
#pragma unroll
    for (int i = 1; i < JOIN_W; ++i) {
        const float4 x = s_sum[warp][i][lane];
        t.x += x.x; t.y += x.y; t.z += x.z; t.w += x.w;
    }
    finish(long_u, long_row, c, t);
}

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename I, typename T, typename Y>
cudaError_t run_embed(const EmbedArgs& x, cudaStream_t s) {
    const bool vec = x.D % 8 == 0 && al16(x.table) && al16(x.out);
    const int per = vec ? 8 : 4, cols = (x.D + per - 1) / per;
    const int tx = std::min(256, (cols + 31) / 32 * 32), ty = 256 / tx;
    const int slabs = (x.D + per * tx - 1) / (per * tx);
    const int64_t each = (int64_t)ty * embed_batch<T>();
    const dim3 grid((unsigned)((x.n + each - 1) / each), slabs);
    return launch_after(vec ? embed_kernel<I, T, Y, true> : embed_kernel<I, T, Y, false>, grid, dim3(tx, ty), 0, 1, s, x.n,
                        x.V, x.D, (const I*)x.ids, (const T*)x.table, x.scale, (Y*)x.out);
}

template <typename I>
cudaError_t embed_ids(const EmbedArgs& x, cudaStream_t s) {
    if (x.dtype == SN_DTYPE_F32)
        return x.out_dtype == SN_DTYPE_F32 ? run_embed<I, float, float>(x, s)
                                           : run_embed<I, float, bf16>(x, s);
    return x.out_dtype == SN_DTYPE_F32 ? run_embed<I, bf16, float>(x, s)
                                       : run_embed<I, bf16, bf16>(x, s);
}

int64_t r256(int64_t x) { return (x + 255) / 256 * 256; }

// CTAs of the sort: what more CTAs save in counting and placing they cost in
// barriers (65536 tokens, 65536 rows: 46 us with 8 and 37 with 16 for the whole
// gradient of 8 columns; 8192: 23 and 25).  A cluster has at most 16, or 8 where
// the device has no room for more.
int sort_ctas(int n) { return n <= 2048 ? 1 : n < 32768 ? 8 : MAX_SORT_CTAS; }

// Items of a unit: 64 where that still gives every SM 16 units (262144 tokens,
// 32000 x 1024: 257 us with 32, 218 with 64, 224 with 128), fewer for small
// problems, but not so few that most rows cross units.
int items_per_unit(int64_t n, int64_t V) {
    return (int)std::max<int64_t>(16, std::min<int64_t>(MAX_IPU, (n + V) / (152 * 16)));
}
int64_t units_for(int64_t n, int64_t V) {
    const int64_t ipu = items_per_unit(n, V);
    return (n + V + ipu - 1) / ipu;
}

template <typename T, typename Y>
cudaError_t run_sums(const SumArgs& a, cudaStream_t s) {
    const bool vec = a.D % 8 == 0 && al16(a.g) && al16(a.out);
    const int cols = (a.D + 7) / 8;
    const int tx = std::min(SUM_T, (cols + 31) / 32 * 32), ty = SUM_T / tx;
    const dim3 grid((a.units + ty - 1) / ty, (a.D + 8 * tx - 1) / (8 * tx));
    const cudaError_t e = launch_after(vec ? row_sums<T, Y, true> : row_sums<T, Y, false>, grid, dim3(tx, ty), 0, 1, s, a);
    if (e != cudaSuccess) return e;
    const int64_t slabs = (a.D + JOIN_COLS - 1) / JOIN_COLS;
    const int per_warp = (int)std::max<int64_t>(1, a.units * slabs / (152 * 64));
    const int64_t warps = (a.units + per_warp - 1) / per_warp * slabs;
    return launch_after(a.n / 4 >= a.V ? join_rows<Y, true> : join_rows<Y, false>,
                        (unsigned)((warps + JOIN_W - 1) / JOIN_W), JOIN_T, 0, 1, s, a, per_warp);
}

}  // namespace

cudaError_t launch_embed(const EmbedArgs& x, cudaStream_t s) {
    return x.ids_type == SN_INDEX_I32 ? embed_ids<int32_t>(x, s) : embed_ids<int64_t>(x, s);
}

int64_t embed_bwd_ws_bytes(int n, int V, int D) {
    const int64_t units = units_for(n, V);
    return 2 * r256((int64_t)n * 8) + 2 * r256(std::min<int64_t>(units, n) * D * 4) +
           3 * r256(units * 4);
}

cudaError_t launch_embed_backward(const EmbedBwdArgs& x, void* ws, cudaStream_t s) {
    char* p = static_cast<char*>(ws);
    const int64_t part = r256((int64_t)x.n * 8), units = units_for(x.n, x.V);
    if (units > INT32_MAX) return cudaErrorInvalidValue;
    SortArgs q{};
    q.n = x.n;
    q.V = x.V;
    int bits = 1;
    while (bits < 31 && (x.V >> bits) != 0) ++bits;    // keys are 0 .. V
    q.passes = (bits + 8) / 9;
    q.bits = (bits + q.passes - 1) / q.passes;
    q.ids = x.ids;
    for (int i = 0; i < 2; ++i) q.entry[i] = (int2*)(p + i * part);
    p += 2 * part;
    const void* k = x.ids_type == SN_INDEX_I32 ? (const void*)sort_kernel<int32_t> : (const void*)sort_kernel<int64_t>;
    cudaError_t e = set_smem_attr_once(k, SORT_SMEM);
    if (e != cudaSuccess) return e;
    int ctas = sort_ctas(x.n);
    if (ctas > 8) {
        bool fits = false;
        e = large_cluster_once(k, SORT_T, SORT_SMEM, ctas, &fits);
        if (e != cudaSuccess) return e;
        if (!fits) ctas = 8;
    }
    e = launch_after(x.ids_type == SN_INDEX_I32 ? sort_kernel<int32_t> : sort_kernel<int64_t>, ctas, SORT_T, SORT_SMEM, ctas,
                     s, q);
    if (e != cudaSuccess) return e;
    SumArgs a{};
    a.n = x.n;
    a.V = x.V;
    a.D = x.D;
    a.ipu = items_per_unit(x.n, x.V);
    a.units = (int)units;
    a.accumulate = x.accumulate;
    a.entry = q.entry[q.passes & 1];
    a.g = x.grad_out;
    a.scale = x.scale;
    a.out = x.grad_table;
    a.tail = (float*)p;
    const int64_t slots = r256(std::min<int64_t>(units, x.n) * x.D * 4);
    a.by_token = units > x.n;
    a.head = (float*)(p + slots);
    a.head_row = (int*)(p + 2 * slots);
    a.tail_row = (int*)(p + 2 * slots + r256(units * 4));
    a.tail_slot = (int*)(p + 2 * slots + 2 * r256(units * 4));
    if (x.dtype == SN_DTYPE_F32)
        return x.grad_dtype == SN_DTYPE_F32 ? run_sums<float, float>(a, s) : run_sums<float, bf16>(a, s);
    return x.grad_dtype == SN_DTYPE_F32 ? run_sums<bf16, float>(a, s) : run_sums<bf16, bf16>(a, s);
}

}  // namespace sn
