// Routing of tokens to experts: the plan (a stable counting sort of the entries by expert) and the
// products with the routing matrix R (tokens x slots, one entry per used slot), its transpose and the
// gradient on its pattern.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "seq_rows.cuh"

namespace sla {
namespace {

constexpr int MAX_EXPERTS = 4096;

// ------------------------------------------------------------------ sort
// A stable counting sort.  A block takes its run of entries in tiles; in a tile warp w owns 32 IT
// consecutive entries and counts them by expert in cnt[w][.] as it goes: equal experts among 32 lanes are
// ranked by lane (votes), so an entry's rank within its warp and expert follows the order of the numbers.
// Prefix sums over the warps, the tiles and (k_route_place) the blocks turn ranks into slots.
//
// Up to one tile of entries (8192 at 256 experts) one block does all of it in one launch.  Above, blocks rank
// their runs and leave histograms, and a second launch adds what lies in front: two launches of up
// to 148 blocks, each a pass over the ids.  Latency bounds it, not memory (131072 x 8 ids: 17 MB, 2.6 us):
// 18 us there, 11 us for 8192 entries, 3.2 us for 64.  Votes over the expert's bits rank a warp in 21 us where
// match_any took 25; entries written from the order in shared memory 18 where scattered ones took 21.
constexpr int ST = 1024;                      // threads at most
constexpr int IT = 8;                         // entries of a lane in a tile
constexpr int SORTED = ST * IT;               // entries that a block puts in order in shared memory

template <typename I>
__device__ __forceinline__ int expert_of(I v, int n_experts)
{
    return v >= 0 && v < (I)n_experts ? (int)v : -1;
}

// off[0 .. n] = exclusive sums of cnt rounded up to `align` (all threads of the block)
__device__ __forceinline__ void padded_offsets(int n, int align, const int *cnt, int *off)
{
    __shared__ int s_warp[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int per = (n + blockDim.x - 1) / blockDim.x, e0 = min(n, (int)threadIdx.x * per), e1 = min(n, e0 + per);
    int sum = 0;
    for (int e = e0; e < e1; ++e)
        sum += (cnt[e] + align - 1) / align * align;
    int inc = sum;
    for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d)
            inc += o;
    }
    if (lane == 31)
        s_warp[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int w = lane < warps ? s_warp[lane] : 0;
        for (int d = 1; d < 32; d *= 2) {
            const int o = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d)
                w += o;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    int at = inc - sum + (warp ? s_warp[warp - 1] : 0);
    for (int e = e0; e < e1; ++e) {
        off[e] = at;
        at += (cnt[e] + align - 1) / align * align;
    }
    if (e1 == n && (e0 < n || threadIdx.x == 0))
        off[n] = at;
    __syncthreads();
}

// offsets, counts and the -1 of slots without an entry, shared out over `parts` blocks
__device__ __forceinline__ void write_plan(int n_experts, int align, int64_t n_slots, const int *cnt,
                                           const int *off, int part, int parts, int32_t *offsets, int32_t *counts, int32_t *entry)
{
    if (part == 0) {
        for (int e = threadIdx.x; e <= n_experts; e += blockDim.x)
            offsets[e] = off[e];
        for (int e = threadIdx.x; e < n_experts; e += blockDim.x)
            counts[e] = cnt[e];
    }
    // a thread an expert where padding is short, a warp where it is long
    const int lanes = align > 16 ? 32 : 1, lane = threadIdx.x & (lanes - 1);
    const int64_t t = (int64_t)part * blockDim.x + threadIdx.x;
    if (align > 1)
        for (int64_t e = t / lanes; e < n_experts; e += (int64_t)parts * blockDim.x / lanes)
            for (int64_t p = (int64_t)off[e] + cnt[e] + lane; p < off[e + 1]; p += lanes)
                entry[p] = -1;
    for (int64_t p = off[n_experts] + (int64_t)part * blockDim.x + threadIdx.x; p < n_slots; p += (int64_t)parts * blockDim.x)
        entry[p] = -1;
}

// Shared memory: per-warp counts (16 bits: a tile has at most 8192 entries), two arrays of sums, the offsets, and for
// one block alone with more than 1024 entries those in order.
static inline int sort_warps(int n_experts) { return std::max(1, std::min(ST / 32, (128 << 10) / (2 * n_experts))); }
static inline size_t sort_smem(int n_experts, int warps, bool staged)
{
    return ((size_t)warps * n_experts * 2 + 15) / 16 * 16 + sizeof(int) * (3 * (size_t)n_experts + 1) +
           (staged ? sizeof(int) * ((size_t)n_experts + 1 + SORTED) : 0);
}

template <typename I, bool ALONE>
__global__ void __launch_bounds__(ST)
    k_route_rank(int64_t n, int64_t per_block, int turns, int n_experts, int align, const I *ids, int64_t n_slots, int32_t *offsets,
                 int32_t *counts, int32_t *entry, int32_t *slot, int32_t *hist)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const size_t cells = (size_t)warps * n_experts;
    uint16_t *cnt = reinterpret_cast<uint16_t *>(smem);
    int *run = reinterpret_cast<int *>(smem + (cells * 2 + 15) / 16 * 16);   // entries of the expert in earlier tiles
    int *sum = run + n_experts;                                             // ... up to this tile
    int *off = sum + n_experts;
    int *front = off + n_experts + 1;
    uint32_t *sorted = reinterpret_cast<uint32_t *>(front + n_experts + 1);
    const int64_t b0 = min(n, per_block * blockIdx.x), b1 = min(n, b0 + per_block);
    const int bits = 32 - __clz(n_experts);
    for (int e = threadIdx.x; e < n_experts; e += blockDim.x)
        run[e] = sum[e] = 0;
    for (int64_t tile = b0; tile < b1 || (ALONE && tile == b0); tile += (int64_t)warps * 32 * turns) {
        const int64_t e0 = tile + (int64_t)warp * 32 * turns + lane;
        int x[IT], rank[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i)
            x[i] = i < turns && e0 + 32 * i < b1 ? expert_of(ids[e0 + 32 * i], n_experts) : -2;
        for (size_t i = threadIdx.x; i < (cells + 7) / 8; i += blockDim.x)
            reinterpret_cast<uint4 *>(cnt)[i] = make_uint4(0, 0, 0, 0);
        __syncthreads();
        uint16_t *mine = cnt + (size_t)warp * n_experts;
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            if (i >= turns)
                break;
            // lanes of the same expert: a vote for each bit (dropped entries and lanes without one count as one more)
            unsigned peers = 0xffffffffu;
            const int key = x[i] < 0 ? n_experts : x[i];
            for (int b = 0; b < bits; ++b) {
                const unsigned set = __ballot_sync(0xffffffffu, key >> b & 1);
                peers &= key >> b & 1 ? set : ~set;
            }
            const int before = x[i] >= 0 ? mine[x[i]] : 0;
            rank[i] = before + __popc(peers & ((1u << lane) - 1));
            __syncwarp();
            if (x[i] >= 0 && (peers >> lane) == 1)     // the last of its kind
                mine[x[i]] = (uint16_t)(before + __popc(peers));
            __syncwarp();
        }
        __syncthreads();
        for (int e = threadIdx.x; e < n_experts; e += blockDim.x) {
            int acc = 0;
#pragma unroll 8
            for (int w = 0; w < warps; ++w) {
                const int c = cnt[(size_t)w * n_experts + e];
                cnt[(size_t)w * n_experts + e] = (uint16_t)acc;
                acc += c;
            }
            run[e] = sum[e];
            sum[e] += acc;
        }
        __syncthreads();
        // Alone, entries of one expert are put next to one another first (k_route_place has the reason).
        const bool staged = ALONE && n > 1024;
        if constexpr (ALONE) {
            padded_offsets(n_experts, align, sum, off);
            if (staged)
                padded_offsets(n_experts, 1, sum, front);
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int64_t e = e0 + 32 * i;
            if (x[i] >= 0) {
                const int p = (ALONE ? off[x[i]] : run[x[i]]) + mine[x[i]] + rank[i];
                slot[e] = p;
                if (staged)
                    sorted[front[x[i]] + p - off[x[i]]] = (uint32_t)x[i] << 16 | (uint32_t)e;
                else if (ALONE)
                    entry[p] = (int)e;
            } else if (x[i] == -1)
                slot[e] = -1;
        }
        __syncthreads();
    }
    if (ALONE && n > 1024)
        for (int q = threadIdx.x; q < front[n_experts]; q += blockDim.x) {
            const int x = (int)(sorted[q] >> 16);
            entry[off[x] + q - front[x]] = (int)(sorted[q] & 0xffffu);
        }
    if constexpr (ALONE)
        write_plan(n_experts, align, n_slots, sum, off, 0, 1, offsets, counts, entry);
    else
        for (int e = threadIdx.x; e < n_experts; e += blockDim.x)
            hist[(size_t)blockIdx.x * n_experts + e] = sum[e];
}

// Ranks within a block's run -> slots.
template <typename I>
__global__ void __launch_bounds__(ST)
    k_route_place(int64_t n, int64_t per_block, int n_experts, int align, const I *ids, int64_t n_slots,
                  int32_t *offsets, int32_t *counts, int32_t *entry, int32_t *slot, const int32_t *hist)
{
    extern __shared__ __align__(16) unsigned char smem[];
    int *cnt = reinterpret_cast<int *>(smem), *base = cnt + n_experts, *off = base + n_experts, *front = off + n_experts + 1;
    uint32_t *sorted = reinterpret_cast<uint32_t *>(front + n_experts + 1);   // (expert, entry of the block) by expert
    const int64_t b0 = min(n, per_block * blockIdx.x), b1 = min(n, b0 + per_block);
    // totals and what lies in front, `parts` threads an expert
    const int parts = max(1, (int)blockDim.x / n_experts);
    for (int e = threadIdx.x; e < n_experts; e += blockDim.x)
        cnt[e] = base[e] = 0;
    __syncthreads();
    if ((int)threadIdx.x < parts * n_experts || parts == 1)
        for (int e = threadIdx.x % (parts == 1 ? blockDim.x : (unsigned)n_experts); e < n_experts; e += blockDim.x) {
            const int part = parts == 1 ? 0 : threadIdx.x / n_experts;
            int all = 0, front = 0;
#pragma unroll 8
            for (int g = part; g < (int)gridDim.x; g += parts) {
                const int v = hist[(size_t)g * n_experts + e];
                all += v;
                front += g < (int)blockIdx.x ? v : 0;
            }
            atomicAdd(&cnt[e], all);                    // whole numbers: any order gives the same sums
            atomicAdd(&base[e], front);
        }
    __syncthreads();
    padded_offsets(n_experts, align, cnt, off);
    const bool one_tile = per_block <= SORTED;
    if (one_tile)
        padded_offsets(n_experts, 1, hist + (size_t)blockIdx.x * n_experts, front);
    for (int e = threadIdx.x; e < n_experts; e += blockDim.x)
        base[e] += off[e];
    __syncthreads();
    for (int64_t t = b0 + threadIdx.x; t < b1; t += (int64_t)blockDim.x * IT) {
        int x[IT], r[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int64_t e = t + (int64_t)i * blockDim.x;
            x[i] = e < b1 ? expert_of(ids[e], n_experts) : -1;
            r[i] = e < b1 ? slot[e] : 0;
        }
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int64_t e = t + (int64_t)i * blockDim.x;
            if (x[i] >= 0) {
                const int p = base[x[i]] + r[i];
                slot[e] = p;
                if (one_tile)
                    sorted[front[x[i]] + r[i]] = (uint32_t)x[i] << 16 | (uint32_t)(e - b0);
                else
                    entry[p] = (int)e;
            }
        }
    }
    // entries of one expert next to one another, so that neighbouring threads write neighbouring slots
    if (one_tile) {
        __syncthreads();
        for (int q = threadIdx.x; q < front[n_experts]; q += blockDim.x) {
            const int x = (int)(sorted[q] >> 16);
            entry[base[x] + q - front[x]] = (int)(b0 + (sorted[q] & 0xffffu));
        }
    }
    write_plan(n_experts, align, n_slots, cnt, off, blockIdx.x, gridDim.x, offsets, counts, entry);
}

// Lets a kernel have the shared memory of the largest call, once per device.  The limit belongs to the process, and calls may
// be made at the same time: one that set its own size could lower another's between that one's set and its launch.
template <auto KERNEL>
static sla_status allow_smem(size_t most)
{
    static std::atomic<uint64_t> ready{0};                 // devices whose limit is set
    int dev = 0;
    SLA_CUDA_TRY(cudaGetDevice(&dev));
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        SLA_CUDA_TRY(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most));
        if (dev < 64)
            ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    return SLA_SUCCESS;
}
static inline size_t place_smem(int n_experts) { return sizeof(int) * (4 * (size_t)n_experts + 2 + SORTED); }

// Blocks of the two-launch sort: a tile each at least, at most 148 (a B200's SMs; a constant, for the workspace's size is
// asked without a device), and histograms of 64 Ki numbers at most, since every block of the second launch reads
// them all.
static inline int64_t sort_blocks(int64_t n, int n_experts)
{
    const int64_t tile = (int64_t)sort_warps(n_experts) * 32 * IT;
    return std::max<int64_t>(1, std::min<int64_t>({(n + tile - 1) / tile, (int64_t)148, (int64_t)65536 / n_experts}));
}

// ------------------------------------------------------------------ products
// One group of G threads a token, a row cut into units of U values (16 bytes where all rows are aligned to
// it).  A token's row crosses memory once: read and written to each of its slots, or summed from them;
// the gradient on the pattern is the dot product of the rows that pass anyway.  Sums run over j in
// order and over the channels in an order fixed by the sizes and the rows' alignment, so results do not
// depend on scheduling.
//
// Memory bounds all four: 16384 tokens x 2 choices x 4096 bf16 take 70 us for R^T x (0.88 of the copy rate on 403 MB),
// 74 for R y (0.84), 111 and 102 with the gradient on the pattern (0.93, 0.80).  What carried them: 16-byte units,
// KU x NV of them in flight a thread, the plan's slots and weights once a thread, up to four turns a
// thread (one turn: R y 87 us), K sums shared out over the lanes (K butterflies: 134 us for R y with its gradient),
// kernels without dot products apart (38 registers instead of 128: R^T x 100 us before).  Rows not aligned
// to 4 bytes go value by value: 4097 channels, R^T x 135 us, R y 178.
constexpr int PT = 256;

template <typename S, int U>
struct Unit {
    using A = typename RowType<S>::A;
    static constexpr int BYTES = U * (int)sizeof(S);
    using Raw = std::conditional_t<BYTES == 16, uint4,
                                   std::conditional_t<BYTES == 8, uint2, std::conditional_t<BYTES == 4, unsigned, uint16_t>>>;
    Raw raw;
    __device__ __forceinline__ void load(const S *p, int left)
    {
        if (U == 1 || left >= U)
            raw = __ldg(reinterpret_cast<const Raw *>(p));
        else if constexpr (U > 1) {
            S s[U];
#pragma unroll
            for (int e = 0; e < U; ++e)
                s[e] = e < left ? p[e] : S(0.0f);
            memcpy(&raw, s, BYTES);
        }
    }
    __device__ __forceinline__ void store(S *p, int left) const
    {
        if (U == 1 || left >= U)
            *reinterpret_cast<Raw *>(p) = raw;
        else if constexpr (U > 1) {
            S s[U];
            memcpy(s, &raw, BYTES);
#pragma unroll
            for (int e = 0; e < U; ++e)
                if (e < left)
                    p[e] = s[e];
        }
    }
    __device__ __forceinline__ void zero() { memset(&raw, 0, BYTES); }
    __device__ __forceinline__ void up(A (&x)[U]) const
    {
        if constexpr (BYTES == 16)
            unpack16(raw, x, S());
        else {
            S s[U];
            memcpy(s, &raw, BYTES);
#pragma unroll
            for (int e = 0; e < U; ++e)
                x[e] = RowType<S>::up(s[e]);
        }
    }
    __device__ __forceinline__ void set(const A (&x)[U])
    {
        if constexpr (BYTES == 16)
            raw = pack16(x, S());
        else {
            S s[U];
#pragma unroll
            for (int e = 0; e < U; ++e)
                s[e] = RowType<S>::down(x[e]);
            memcpy(&raw, s, BYTES);
        }
    }
};

template <typename S>
struct RouteArgs {
    using A = typename RowType<S>::A;
    int64_t n_tokens, n_slots, n_chan;
    int top_k, n_experts, fill, fill_blocks;
    const int32_t *offsets, *counts, *slot;
    const A *weight;
    const S *tok;             // token side, read: x, dy
    const S *slt;             // slot side, read: ys, dxs
    S *tok_out, *slt_out;
    int64_t ldtok, ldslt, ldtok_out, ldslt_out;
    A *dweight;
};

// Sums of K values (a power of two) over a group of G threads (a power of two, a warp at least), in a fixed
// order; the j-th ends in the group's j-th thread.  Within a warp the lanes first share the values out, each exchange
// halving the number a lane carries (K - 1 + 5 - log2 K exchanges instead of 5 K).
template <typename A, int K>
__device__ __forceinline__ A group_sums(A (&d)[K], int G, A (*s_red)[K])
{
    const int lane = threadIdx.x & 31;
    int bit = 1;
#pragma unroll
    for (int n = K / 2; n > 0; n /= 2, bit *= 2) {
        const bool upper = lane & bit;
#pragma unroll
        for (int j = 0; j < n; ++j) {
            const A send = upper ? d[j] : d[j + n], keep = upper ? d[j + n] : d[j];
            d[j] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
        }
    }
    for (; bit < 32; bit *= 2)
        d[0] += __shfl_xor_sync(0xffffffffu, d[0], bit);
    // the lane whose low bits, read from the lowest up, spell j from its highest bit down has value j
    int at = 0;
#pragma unroll
    for (int n = K / 2, b = 1; n > 0; n /= 2, b *= 2)
        at |= (lane & n) ? b : 0;
    if (G == 32)
        return __shfl_sync(0xffffffffu, d[0], at);
    const int warp = threadIdx.x >> 5, first = (threadIdx.x & ~(G - 1)) >> 5, j = threadIdx.x & (G - 1);
    const A mine = __shfl_sync(0xffffffffu, d[0], at);
    __syncthreads();
    if (lane < K)
        s_red[warp][lane] = mine;
    __syncthreads();
    A t = A(0);
    if (j < K)
        for (int w = 0; w < G / 32; ++w)
            t += s_red[first + w][j];
    return t;
}

// Zeros in the slots without an entry, a row a warp: block f of the fill blocks takes the padding rows r of
// expert e with (e + r) % fill_blocks = f, and its share of the rest.
template <typename S, int U>
__device__ __forceinline__ void fill_blanks(const RouteArgs<S> &g, int f)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nf = g.fill_blocks;
    const int64_t nunits = (g.n_chan + U - 1) / U;
    Unit<S, U> z;
    z.zero();
    auto clear = [&](int64_t row) {
        S *p = g.slt_out + row * g.ldslt_out;
        for (int64_t u = lane; u < nunits; u += 32)
            z.store(p + u * U, (int)min((int64_t)U, g.n_chan - u * U));
    };
    for (int e0 = warp * 32; e0 < g.n_experts; e0 += PT) {
        const int e = e0 + lane;
        int64_t r0 = 0, n = 0;
        if (e < g.n_experts) {
            r0 = min(max((int64_t)g.offsets[e] + g.counts[e], (int64_t)0), g.n_slots);
            n = min((int64_t)g.offsets[e + 1], g.n_slots) - r0;
        }
        const int first = (f + nf - e % nf) % nf;
        for (unsigned has = __ballot_sync(0xffffffffu, first < n); has; has &= has - 1) {
            const int l = __ffs(has) - 1;
            const int64_t q0 = __shfl_sync(0xffffffffu, r0, l), m = __shfl_sync(0xffffffffu, n, l);
            for (int64_t r = __shfl_sync(0xffffffffu, first, l); r < m; r += nf)
                clear(q0 + r);
        }
    }
    if (g.fill)
        for (int64_t r = max((int64_t)g.offsets[g.n_experts], (int64_t)0) + (int64_t)f * (PT / 32) + warp; r < g.n_slots;
             r += (int64_t)nf * (PT / 32))
            clear(r);
}

// The slots and weights of choices j0 .. j0 + KU of a token; -1 where there is none.
template <typename S, int KU>
struct Choices {
    using A = typename RowType<S>::A;
    int p[KU];
    A w[KU];
    __device__ __forceinline__ void load(const RouteArgs<S> &g, int64_t t, int j0, bool live)
    {
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            const bool has = live && j0 + j < g.top_k;
            p[j] = has ? g.slot[t * g.top_k + j0 + j] : -1;
            if (p[j] >= g.n_slots)
                p[j] = -1;
            w[j] = has && g.weight ? g.weight[t * g.top_k + j0 + j] : A(1);
        }
    }
};

// R^T x, and with DW x . ys on the pattern.  KU choices and NV units at a time.
template <typename S, int U, int KU, int NV, bool DW>
__global__ void __launch_bounds__(PT) k_route_to_slots(const __grid_constant__ RouteArgs<S> g, int G)
{
    using A = typename RowType<S>::A;
    __shared__ A s_red[PT / 32][KU];
    if ((int)blockIdx.x < g.fill_blocks) {
        fill_blanks<S, U>(g, blockIdx.x);
        return;
    }
    const int64_t t = (int64_t)(blockIdx.x - g.fill_blocks) * (PT / G) + threadIdx.x / G;
    const int lane = threadIdx.x & (G - 1);
    const bool live = t < g.n_tokens;
    const int nunits = live ? (int)((g.n_chan + U - 1) / U) : 0;
    const S *x = g.tok + (live ? t : 0) * g.ldtok;
    for (int j0 = 0; j0 < g.top_k; j0 += KU) {
        Choices<S, KU> ch;
        ch.load(g, t, j0, live);
        A dot[KU];
#pragma unroll
        for (int j = 0; j < KU; ++j)
            dot[j] = A(0);
        for (int u0 = lane; u0 < nunits; u0 += G * NV) {
            Unit<S, U> v[NV], o[DW ? KU : 1][NV];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(u0 + i * G) * U;
                if (u0 + i * G < nunits)
                    v[i].load(x + c, (int)min((int64_t)U, g.n_chan - c));
                else
                    v[i].zero();
                if constexpr (DW) {
#pragma unroll
                    for (int j = 0; j < KU; ++j) {
                        if (ch.p[j] >= 0 && u0 + i * G < nunits)
                            o[j][i].load(g.slt + ch.p[j] * g.ldslt + c, (int)min((int64_t)U, g.n_chan - c));
                        else
                            o[j][i].zero();
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(u0 + i * G) * U;
                if (u0 + i * G >= nunits)
                    continue;
                const int left = (int)min((int64_t)U, g.n_chan - c);
                A f[U];
                if (DW || g.weight)
                    v[i].up(f);
                if constexpr (DW) {
#pragma unroll
                    for (int j = 0; j < KU; ++j) {
                        A y[U];
                        o[j][i].up(y);
                        if (ch.p[j] >= 0)
#pragma unroll
                            for (int e = 0; e < U; ++e)
                                dot[j] = fma_of(f[e], y[e], dot[j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < KU; ++j) {
                    if (ch.p[j] < 0)
                        continue;
                    Unit<S, U> r = v[i];
                    if (g.weight) {
                        A y[U];
#pragma unroll
                        for (int e = 0; e < U; ++e)
                            y[e] = ch.w[j] * f[e];
                        r.set(y);
                    }
                    r.store(g.slt_out + ch.p[j] * g.ldslt_out + c, left);
                }
            }
        }
        if constexpr (DW) {
            const A sum = group_sums<A, KU>(dot, G, s_red);
            if (live && lane < KU && j0 + lane < g.top_k)
                g.dweight[t * g.top_k + j0 + lane] = sum;
        }
    }
}

// R ys, and with DW x . ys on the pattern: in the same pass with up to KU choices, after the sums with more.
template <typename S, int U, int KU, int NV, bool DW>
__global__ void __launch_bounds__(PT) k_route_to_tokens(const __grid_constant__ RouteArgs<S> g, int G)
{
    using A = typename RowType<S>::A;
    __shared__ A s_red[PT / 32][KU];
    const int64_t t = (int64_t)blockIdx.x * (PT / G) + threadIdx.x / G;
    const int lane = threadIdx.x & (G - 1);
    const bool live = t < g.n_tokens;
    const int nunits = live ? (int)((g.n_chan + U - 1) / U) : 0;
    const bool one = g.top_k <= KU;
    Choices<S, KU> ch;
    ch.load(g, t, 0, live);
    A dot[KU];
#pragma unroll
    for (int j = 0; j < KU; ++j)
        dot[j] = A(0);
    const S *x = DW ? g.tok + (live ? t : 0) * g.ldtok : nullptr;
    for (int u0 = lane; u0 < nunits; u0 += G * NV) {
        A acc[NV][U];
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < U; ++e)
                acc[i][e] = A(0);
        for (int j0 = 0; j0 < g.top_k; j0 += KU) {
            if (!one)
                ch.load(g, t, j0, live);
            Unit<S, U> o[KU][NV], v[DW ? NV : 1];
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int64_t c = (int64_t)(u0 + i * G) * U;
                const bool in = u0 + i * G < nunits;
                const int left = (int)min((int64_t)U, g.n_chan - c);
#pragma unroll
                for (int j = 0; j < KU; ++j) {
                    if (ch.p[j] >= 0 && in)
                        o[j][i].load(g.slt + ch.p[j] * g.ldslt + c, left);
                    else
                        o[j][i].zero();
                }
                if constexpr (DW) {
                    v[i].zero();
                    if (one && in)
                        v[i].load(x + c, left);
                }
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                A f[U];
                if constexpr (DW)
                    v[i].up(f);
#pragma unroll
                for (int j = 0; j < KU; ++j) {
                    if (ch.p[j] < 0)
                        continue;
                    A y[U];
                    o[j][i].up(y);
#pragma unroll
                    for (int e = 0; e < U; ++e) {
                        if constexpr (DW)
                            dot[j] = fma_of(f[e], y[e], dot[j]);
                        acc[i][e] = fma_of(ch.w[j], y[e], acc[i][e]);
                    }
                }
            }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int64_t c = (int64_t)(u0 + i * G) * U;
            if (u0 + i * G >= nunits)
                continue;
            Unit<S, U> r;
            r.set(acc[i]);
            r.store(g.tok_out + t * g.ldtok_out + c, (int)min((int64_t)U, g.n_chan - c));
        }
    }
    if constexpr (DW) {
        for (int j0 = 0; j0 < g.top_k; j0 += KU) {
            if (!one) {
                ch.load(g, t, j0, live);
#pragma unroll
                for (int j = 0; j < KU; ++j)
                    dot[j] = A(0);
                for (int u = lane; u < nunits; u += G) {
                    const int64_t c = (int64_t)u * U;
                    const int left = (int)min((int64_t)U, g.n_chan - c);
                    Unit<S, U> v;
                    v.load(x + c, left);
                    A f[U], y[U];
                    v.up(f);
#pragma unroll
                    for (int j = 0; j < KU; ++j)
                        if (ch.p[j] >= 0) {
                            v.load(g.slt + ch.p[j] * g.ldslt + c, left);
                            v.up(y);
#pragma unroll
                            for (int e = 0; e < U; ++e)
                                dot[j] = fma_of(f[e], y[e], dot[j]);
                        }
                }
            }
            const A sum = group_sums<A, KU>(dot, G, s_red);
            if (live && lane < KU && j0 + lane < g.top_k)
                g.dweight[t * g.top_k + j0 + lane] = sum;
        }
    }
}

// Threads a token, a warp at least and a block at most: its units NV at a time, in up to four turns where there
// are tokens enough to fill the GPU's threads all the same (fewer threads a token spend less on its plan and
// on the sums over the group).
static inline int group_of(int64_t n_tokens, int64_t n_chan, int U, int NV)
{
    const int64_t nunits = (n_chan + U - 1) / U;
    for (int turns = 4;; turns /= 2) {
        int G = 32;
        while (G < PT && (int64_t)G * NV * turns < nunits)
            G *= 2;
        if (turns == 1 || n_tokens * G >= (int64_t)sm_count() * 2048)
            return G;
    }
}

template <typename S, int U, int KU, int NV, bool DW>
sla_status launch_product(RouteArgs<S> &g, bool to_slots, cudaStream_t s)
{
    const int G = group_of(g.n_tokens, g.n_chan, U, NV);
    const int64_t blocks = (g.n_tokens + PT / G - 1) / (PT / G);
    if (to_slots) {
        // a fill block for every 64 KiB of slot rows that may be blank, at most two an SM
        const int64_t bytes = g.n_slots * g.n_chan * (int64_t)sizeof(S);
        g.fill_blocks = (int)std::max<int64_t>(1, std::min<int64_t>(2 * sm_count(), bytes >> 16));
        k_route_to_slots<S, U, KU, NV, DW><<<(unsigned)(blocks + g.fill_blocks), PT, 0, s>>>(g, G);
    } else if (blocks > 0)
        k_route_to_tokens<S, U, KU, NV, DW><<<(unsigned)blocks, PT, 0, s>>>(g, G);
    SLA_CUDA_TRY(cudaGetLastError());
    return SLA_SUCCESS;
}

template <typename S, int U, int KU, int NV>
sla_status launch_dw(RouteArgs<S> &g, bool to_slots, cudaStream_t s)
{
    return g.dweight ? launch_product<S, U, KU, NV, true>(g, to_slots, s)
                     : launch_product<S, U, KU, NV, false>(g, to_slots, s);
}

// KU choices times NV units in flight a thread, more units where they are short.
template <typename S, int U>
sla_status launch_unit(RouteArgs<S> &g, bool to_slots, cudaStream_t s)
{
    constexpr int M = U * sizeof(S) == 16 ? 1 : U * sizeof(S) > 2 ? 2 : 4;
    if (g.top_k <= 2)
        return launch_dw<S, U, 2, 2 * M>(g, to_slots, s);
    if (g.top_k <= 4)
        return launch_dw<S, U, 4, 2 * M>(g, to_slots, s);
    return launch_dw<S, U, 8, M>(g, to_slots, s);
}

template <typename S>
sla_status run_product(RouteArgs<S> g, bool to_slots, cudaStream_t s)
{
    uintptr_t bits = 0;
    auto see = [&](const void *p, int64_t ld) {
        if (p)
            bits |= (uintptr_t)p | (uintptr_t)(ld * (int64_t)sizeof(S));
    };
    see(g.tok, g.ldtok);
    see(g.slt, g.ldslt);
    see(g.tok_out, g.ldtok_out);
    see(g.slt_out, g.ldslt_out);
    if (bits % 16 == 0)
        return launch_unit<S, 16 / (int)sizeof(S)>(g, to_slots, s);
    if constexpr (sizeof(S) == 2)
        if (bits % 4 == 0)
            return launch_unit<S, 2>(g, to_slots, s);
    return launch_unit<S, 1>(g, to_slots, s);
}

sla_status check_route(int32_t dtype, int64_t n_tokens, int32_t top_k, int64_t n_slots, int64_t n_chan,
                       const int32_t *d_slot)
{
    if (!row_dtype_ok(dtype))
        return fail(SLA_ERR_INVALID_ARG, "dtype must be SLA_F32, SLA_F64, SLA_BF16 or SLA_F16");
    if (n_tokens < 0 || top_k < 1 || n_tokens > INT32_MAX / top_k)
        return fail(SLA_ERR_INVALID_ARG, "top_k must be at least 1 and n_tokens * top_k within [0, 2^31)");
    if (n_slots < 0 || n_slots > INT32_MAX || n_chan < 0 || n_chan > INT32_MAX)
        return fail(SLA_ERR_INVALID_ARG, "slots and channels must be within [0, 2^31)");
    if (n_tokens > 0 && !d_slot)
        return fail(SLA_ERR_INVALID_ARG, "d_slot is NULL");
    return SLA_SUCCESS;
}

sla_status check_rows(const void *p, int64_t ld, int64_t n_rows, int64_t n_chan, bool out)
{
    if (n_rows == 0 || n_chan == 0)
        return SLA_SUCCESS;
    if (!p || (ld < n_chan && (out || ld != 0)))
        return fail(SLA_ERR_INVALID_ARG, "NULL rows, or a row stride below the number of channels");
    return SLA_SUCCESS;
}

sla_status check_plan(int32_t n_experts, const int32_t *d_offsets, const int32_t *d_counts, uint32_t flags)
{
    if (n_experts < 1 || !d_offsets || !d_counts)
        return fail(SLA_ERR_INVALID_ARG, "n_experts must be at least 1 and d_offsets, d_counts not NULL");
    if (flags & ~SLA_FILL_REST)
        return fail(SLA_ERR_INVALID_ARG, "unknown flags");
    return SLA_SUCCESS;
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

size_t sla_route_workspace_bytes(int64_t n_tokens, int32_t top_k, int32_t n_experts)
{
    if (n_tokens <= 0 || top_k < 1 || n_tokens > INT32_MAX / top_k || n_experts < 1 || n_experts > MAX_EXPERTS)
        return 0;
    const int64_t blocks = sort_blocks(n_tokens * top_k, n_experts);
    return blocks > 1 ? sizeof(int32_t) * (size_t)blocks * (size_t)n_experts : 0;
}

sla_status sla_route_sort(int64_t n_tokens, int32_t top_k, int32_t n_experts, int32_t align, const void *d_expert,
                          int32_t id_bytes, int64_t n_slots, int32_t *d_offsets, int32_t *d_counts, int32_t *d_entry,
                          int32_t *d_slot, void *d_work, size_t work_bytes, void *stream)
{
    if (n_tokens < 0 || top_k < 1 || n_tokens > INT32_MAX / top_k)
        return fail(SLA_ERR_INVALID_ARG, "top_k must be at least 1 and n_tokens * top_k within [0, 2^31)");
    if (n_experts < 1 || align < 1)
        return fail(SLA_ERR_INVALID_ARG, "n_experts and align must be at least 1");
    if (n_experts > MAX_EXPERTS)
        return fail(SLA_ERR_UNSUPPORTED, "more than 4096 experts");
    if (id_bytes != 4 && id_bytes != 8)
        return fail(SLA_ERR_INVALID_ARG, "id_bytes must be 4 or 8");
    const int64_t n = n_tokens * top_k;
    if (n_slots < n + (int64_t)n_experts * (align - 1) || n_slots > INT32_MAX)
        return fail(SLA_ERR_INVALID_ARG, "n_slots must be at least n_tokens * top_k + n_experts * (align - 1), below 2^31");
    if (!d_offsets || !d_counts || (n > 0 && (!d_expert || !d_slot)) || (n_slots > 0 && !d_entry))
        return fail(SLA_ERR_INVALID_ARG, "NULL array");
    const size_t need = sla_route_workspace_bytes(n_tokens, top_k, n_experts);
    if (need && (!d_work || work_bytes < need || (uintptr_t)d_work % 16))
        return fail(SLA_ERR_INVALID_ARG, "d_work is NULL, smaller than sla_route_workspace_bytes or not 16-byte aligned");
    cudaStream_t s = (cudaStream_t)stream;
    const int warps = sort_warps(n_experts);
    const int64_t blocks = sort_blocks(n, n_experts);
    const size_t smem = sort_smem(n_experts, warps, blocks == 1 && n > 1024);
    auto run = [&](auto ids) -> sla_status {
        using I = std::remove_const_t<std::remove_pointer_t<decltype(ids)>>;
        if (blocks == 1) {
            // few entries: a lane takes one, as long as there are warps
            const int w = (int)std::min<int64_t>(warps, std::max<int64_t>({1, (n + 31) / 32, ((int64_t)n_experts + 31) / 32}));
            const int turns = (int)std::max<int64_t>(1, (n + 32 * w - 1) / (32 * w));
            SLA_TRY((allow_smem<k_route_rank<I, true>>(sort_smem(MAX_EXPERTS, sort_warps(MAX_EXPERTS), true))));
            k_route_rank<I, true><<<1, 32 * w, smem, s>>>(n, n, turns, n_experts, align, ids, n_slots, d_offsets, d_counts,
                                                         d_entry, d_slot, nullptr);
        } else {
            const int64_t tile = (int64_t)warps * 32 * IT, per = ((n + blocks - 1) / blocks + tile - 1) / tile * tile;
            const unsigned grid = (unsigned)((n + per - 1) / per);
            SLA_TRY((allow_smem<k_route_rank<I, false>>(sort_smem(MAX_EXPERTS, sort_warps(MAX_EXPERTS), false))));
            SLA_TRY(allow_smem<k_route_place<I>>(place_smem(MAX_EXPERTS)));
            k_route_rank<I, false><<<grid, 32 * warps, smem, s>>>(n, per, IT, n_experts, align, ids, n_slots, d_offsets,
                                                                 d_counts, d_entry, d_slot, (int32_t *)d_work);
            SLA_CUDA_TRY(cudaGetLastError());              // the second launch takes the ranks as places to write to
            k_route_place<I><<<grid, ST, place_smem(n_experts), s>>>(n, per, n_experts, align, ids, n_slots, d_offsets, d_counts,
                                                                     d_entry, d_slot, (const int32_t *)d_work);
        }
        SLA_CUDA_TRY(cudaGetLastError());
        return SLA_SUCCESS;
    };
    return id_bytes == 4 ? run((const int32_t *)d_expert) : run((const int64_t *)d_expert);
}

sla_status sla_route_dispatch(int32_t dtype, int64_t n_tokens, int32_t top_k, int32_t n_experts, int64_t n_slots,
                              int64_t n_chan, const void *d_x, int64_t ldx, const int32_t *d_offsets,
                              const int32_t *d_counts, const int32_t *d_slot, const void *d_weight, void *d_xs,
                              int64_t ldxs, uint32_t flags, void *stream)
{
    return sla_route_combine_adjoint(dtype, n_tokens, top_k, n_experts, n_slots, n_chan, d_x, ldx, d_offsets, d_counts,
                                     d_slot, d_weight, nullptr, 0, d_xs, ldxs, nullptr, flags, stream);
}

sla_status sla_route_combine(int32_t dtype, int64_t n_tokens, int32_t top_k, int64_t n_slots, int64_t n_chan,
                             const void *d_ys, int64_t ldys, const int32_t *d_slot, const void *d_weight, void *d_y,
                             int64_t ldy, void *stream)
{
    return sla_route_dispatch_adjoint(dtype, n_tokens, top_k, n_slots, n_chan, d_ys, ldys, d_slot, d_weight, nullptr, 0,
                                      d_y, ldy, nullptr, stream);
}

sla_status sla_route_dispatch_adjoint(int32_t dtype, int64_t n_tokens, int32_t top_k, int64_t n_slots, int64_t n_chan,
                                      const void *d_dxs, int64_t lddxs, const int32_t *d_slot, const void *d_weight,
                                      const void *d_x, int64_t ldx, void *d_dx, int64_t lddx, void *d_dweight,
                                      void *stream)
{
    SLA_TRY(check_route(dtype, n_tokens, top_k, n_slots, n_chan, d_slot));
    if (n_tokens == 0 || (n_chan == 0 && !d_dweight))
        return SLA_SUCCESS;
    SLA_TRY(check_rows(d_dxs, lddxs, n_slots, n_chan, false));
    SLA_TRY(check_rows(d_dx, lddx, n_tokens, n_chan, true));
    if (d_dweight)
        SLA_TRY(check_rows(d_x, ldx, n_tokens, n_chan, false));
    return with_row_type(dtype, [&](auto tag) {
        using S = decltype(tag);
        using A = typename RowType<S>::A;
        RouteArgs<S> g{};
        g.n_tokens = n_tokens;
        g.n_slots = n_slots;
        g.n_chan = n_chan;
        g.top_k = top_k;
        g.slot = d_slot;
        g.weight = (const A *)d_weight;
        g.slt = (const S *)d_dxs;
        g.ldslt = lddxs;
        g.tok_out = (S *)d_dx;
        g.ldtok_out = lddx;
        if (d_dweight) {
            g.tok = (const S *)d_x;
            g.ldtok = ldx;
            g.dweight = (A *)d_dweight;
        }
        return run_product<S>(g, false, (cudaStream_t)stream);
    });
}

sla_status sla_route_combine_adjoint(int32_t dtype, int64_t n_tokens, int32_t top_k, int32_t n_experts,
                                     int64_t n_slots, int64_t n_chan, const void *d_dy, int64_t lddy,
                                     const int32_t *d_offsets, const int32_t *d_counts, const int32_t *d_slot,
                                     const void *d_weight, const void *d_ys, int64_t ldys, void *d_dys, int64_t lddys,
                                     void *d_dweight, uint32_t flags, void *stream)
{
    SLA_TRY(check_route(dtype, n_tokens, top_k, n_slots, n_chan, d_slot));
    SLA_TRY(check_plan(n_experts, d_offsets, d_counts, flags));
    if (n_chan == 0 && !d_dweight)
        return SLA_SUCCESS;
    SLA_TRY(check_rows(d_dy, lddy, n_tokens, n_chan, false));
    SLA_TRY(check_rows(d_dys, lddys, n_slots, n_chan, true));
    if (d_dweight && n_tokens > 0)
        SLA_TRY(check_rows(d_ys, ldys, n_slots, n_chan, false));
    return with_row_type(dtype, [&](auto tag) {
        using S = decltype(tag);
        using A = typename RowType<S>::A;
        RouteArgs<S> g{};
        g.n_tokens = n_tokens;
        g.n_slots = n_slots;
        g.n_chan = n_chan;
        g.top_k = top_k;
        g.n_experts = n_experts;
        g.fill = (flags & SLA_FILL_REST) != 0;
        g.offsets = d_offsets;
        g.counts = d_counts;
        g.slot = d_slot;
        g.weight = (const A *)d_weight;
        g.tok = (const S *)d_dy;
        g.ldtok = lddy;
        g.slt_out = (S *)d_dys;
        g.ldslt_out = lddys;
        if (d_dweight && n_tokens > 0) {
            g.slt = (const S *)d_ys;
            g.ldslt = ldys;
            g.dweight = (A *)d_dweight;
        }
        return run_product<S>(g, true, (cudaStream_t)stream);
    });
}

}  // extern "C"
