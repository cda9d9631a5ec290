// The gated linear recurrence as one pass over the rows (both directions).
//
// Mathematics.  Forward, h_t = a_t h_{t-1} + u_t with u = w b.  Backward, with lambda_t = g_t + a_{t+1}
// lambda_{t+1}, the carried quantity is e_t = a_t lambda_t, so that e_t = a_t (g_t + e_{t+1}) uses its own
// row's coefficient only and h_0's gradient is e of the first row.  A run of rows is an affine
// map of the state that enters it, x -> A x + H (A: product of its coefficients, H: the run's
// result from a zero state), and runs compose by (A2 A1, A2 H1 + H2).
//
// Layout.  A tile is C scan positions (rows in scan order; backward counts from the last row)
// times 128 bytes of channels.  A compute thread owns a run of R = 4 consecutive positions of 16 bytes of channels;
// 8 threads make a row, so the tile has NR = 4 NW runs.  Tiles are taken by ticket, chunk-major, by
// one persistent block per SM.
//
// One block runs these at the same time, tile i being the oldest:
//   pass 1      tile i + 1: the coefficients, kept in registers for pass 2, and each thread's (A, H), left in
//               shared memory;
//   map warps   tile i + 1, one thread a channel, over the runs in order: the tile's (A, H), published for later
//               chunks, and for every run the map of the runs in front of it;
//   state warps tile i + 1: the state that enters it, from what earlier chunks published; its own leaving
//               state, published;
//   pass 2      tile i: the state that enters the run, every row from it in the order of the formula, and the
//               stores;
//   plan warp   the ticket of tile i + 3, the sequence borders in it, and its rows into shared memory by one tensor
//               copy an input (backward, what only pass 2 reads: of tile i + 1).  Where rows are not aligned to
//               16 bytes every compute warp copies its own rows instead, by units of 4 bytes (fp64: 8) or
//               value by value.
// So each input is read once and each gate evaluated once, and the wait on earlier chunks passes while the
// compute warps are at another tile.  They meet once a tile, where they take over the entering states.
//
// Across chunks a channel publishes (A, H) as soon as pass 1 has them, and the state that leaves the
// chunk, x', once it knows the state that enters.  A later chunk goes back to the nearest chunk whose x' is
// there and applies the (A, H) behind it in order.  x' = fma(A, x, H) from the same published
// (A, H) everywhere, so the result does not depend on how far a chunk had to go back, and the same inputs give the
// same bits.  Every word carries its own "not there yet" (all bits set, a NaN that is never published),
// so one relaxed load gets both and no fence is needed.  A tile waits on tiles with lower
// tickets only, whose blocks are running, so the wait ends however many blocks are resident; it
// is bounded all the same, and a chunk that gave up goes on with NaN.
//
// What bounds it.  Memory must carry z, b and h once (backward z, g, h, dz, db): 6 (10) bytes a value in 16
// bits.  The kernel moves little more (376 of 403 MB at 16384 x 4096 bf16, forward, besides 8 + 4 bytes a channel
// and chunk of published words) but runs at 0.59 of the copy rate there, 103 us, 0.65 to 0.69 in fp32 (16384 x 2048, 89 to
// 95 us), backward 0.70 (146 us) and 0.75 (136 us): about 23 instructions a value at 43 % of the issue slots.
// Warps wait for one another's results once a tile and for fixed latencies in between; 16 warps of 128 registers are
// all that fit.  Measured on the way (solve 65536 x 4096 bf16): every gate twice instead of kept coefficients and
// combining runs by shuffles 655 us, maps by the scan warps 532, four scan threads a channel 501, tensor copies, kept
// coefficients and paired arithmetic 455, first states as entering states 424, guards out of line 403 to 414, maps
// published as they are 362 to 385.  Rows of 128 bytes by a bulk copy each took 185 us where tensor copies took 105 (16384 x
// 4096); copies by one warp's cp.async 171; runs of 8 rows by 7 warps 157; two blocks of half a tile an SM 215.  Few
// channels leave few chunks side by side and the chain of chunks bounds: 200000 x 64 bf16 takes 75 us of a floor
// of 12.  Tiles with borders cost half as much again (16384 x 4096 in 100 sequences: 155 us).
//
// A sequence border inside a run makes its map constant.  Such a map is marked by A = -0 (products are
// normalised to +0), because 0 * x would carry a NaN or an infinity across the border.
//
// A channel whose (A, H) is not finite has no map: a coefficient or an input is not, or a product or a sum of the
// tile left the range, although the states themselves may stay in it.  Its rows are read again and taken one
// by one from the state that enters the tile, and later chunks wait for the one that leaves.  A product that
// vanishes counts as 0.  Rows full of NaN need no wait: solve 65536 x 4096 bf16 820 us; coefficients of 2 over
// rows of zeros, whose every tile overflows, take 13.5 ms there.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "seq_rows.cuh"

namespace sla {

// Offsets are read from the device and clamped, so that no offset leads outside the rows.
struct SeqBounds {
    const int32_t *off;   // NULL: equal lengths
    int64_t n_tokens;
    int32_t n_seq;
    __device__ __forceinline__ int64_t at(int64_t s) const
    {
        if (!off)
            return n_seq > 0 ? n_tokens / n_seq * s : 0;
        const int64_t v = off[s];
        return v < 0 ? 0 : v > n_tokens ? n_tokens : v;
    }
};

// Arguments of either direction.  in[0] = z; forward in[1] = b; backward in[1] = dh, in[2] = h, in[3] = b.
// out[0] = h; backward out[0] = db, out[1] = dz.
template <typename S>
struct RecurArgs {
    using A = typename RowType<S>::A;
    SeqBounds q;
    int64_t n_chan;
    int n_chunks, n_cb;        // tiles along the rows and along the channels
    const S *in[4];
    int64_t ldin[4];
    S *out[2];
    int64_t ldout[2];
    const A *enter;            // forward h0, backward dh_last
    const A *before;           // backward: h0
    A *leave;                  // forward h_last, backward dh0
    CUtensorMap map[4];        // of the inputs, where rows go by tensor copies
    int fill;                  // zeros in rows outside every sequence
    unsigned *ticket;          // NULL with one chunk
    unsigned long long *agg;   // [n_chunks][n_chan] words (fp64: two each)
    void *inc;                 // [n_chunks][n_chan] fp32 or fp64
};

template <typename S, int GATE, bool REV>
struct RecurShape {
    static constexpr int NIN = REV ? (GATE == SLA_GATE_SIGMOID ? 4 : 3) : 2;
    static constexpr int V = 16 / (int)sizeof(S);          // channels of a thread
    static constexpr int W = 8 * V;                        // channels of a tile
    static constexpr int R = 4;                            // rows of a run
    static constexpr int N1 = 2;                           // inputs that pass 1 reads; the others wait for pass 2
    // Compute warps: 16 warps of 128 registers in all, or what shared memory allows
    static constexpr int NW = !REV ? 11 : NIN == 3 ? 10 : 9;
    static constexpr int NS = 3;                           // tiles that plan and loads are ahead
    static constexpr int NZ = 2;                           // stages of input 0, done with after pass 1
    static constexpr int N1S = 4;                          // stages of input 1
    static constexpr int NX = 2;                           // stages of the inputs that only pass 2 reads
    static constexpr int NB = 2;                           // tiles between pass 1 and pass 2
    static constexpr int NP = NS + 2;                      // plan slots
    static constexpr int NR = NW * 4;                      // runs
    static constexpr int C = NR * R;
    static constexpr int NC = NW * 32;                     // compute threads
    static constexpr int NK = (W + 31) / 32 * 32;          // map threads, and state threads
    static constexpr int NT = NC + 2 * NK + 32;
};

__device__ __forceinline__ void bar_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void bar_arrive(int id, int n)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}

template <int B>
__device__ __forceinline__ void copy_async(void *dst, const void *src, int bytes)
{
    const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
    if constexpr (B == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(bytes) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(d), "l"(src), "r"(bytes), "n"(B) : "memory");
}

// Barriers in shared memory that copies arrive at.
__device__ __forceinline__ unsigned smem_at(const void *p) { return (unsigned)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void mbar_init(unsigned long long *bar, int count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_at(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(unsigned long long *bar, int bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_at(bar)), "r"(bytes) : "memory");
}
// A box of a tile's rows, from column x (a multiple of 16 bytes) and row y (which may lie in front of the first)
__device__ __forceinline__ void box_in(void *dst, const CUtensorMap *map, int x, int y, unsigned long long *bar)
{
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                     smem_at(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(smem_at(bar))
                 : "memory");
}
__device__ __forceinline__ void mbar_arrive(unsigned long long *bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_at(bar)) : "memory");
}
__device__ __forceinline__ void mbar_arrive_after_copies(unsigned long long *bar)
{
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_at(bar)) : "memory");
}
// Waits for the phase to end, a bounded number of times; false if it did not.
__device__ __forceinline__ bool mbar_wait(unsigned long long *bar, unsigned parity)
{
    for (int i = 0; i < 1 << 22; ++i) {
        unsigned done;
        asm volatile("{ .reg .pred p;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p; }"
                     : "=r"(done)
                     : "r"(smem_at(bar)), "r"(parity)
                     : "memory");
        if (done)
            return true;
    }
    return false;
}

// ------------------------------------------------------------------ affine maps
__device__ __forceinline__ bool is_const(float a) { return __float_as_uint(a) == 0x80000000u; }
__device__ __forceinline__ bool is_const(double a) { return (unsigned long long)__double_as_longlong(a) == 0x8000000000000000ull; }
template <typename A>
__device__ __forceinline__ A const_mark() { return A(-0.0); }
// x -> A x + H at x
template <typename A>
__device__ __forceinline__ A apply(A a, A x, A h)
{
    return is_const(a) ? h : fma_of(a, x, h);
}

// ------------------------------------------------------------------ published words
__device__ __forceinline__ unsigned long long ld_word(const unsigned long long *p)
{
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ unsigned ld_word(const unsigned *p)
{
    unsigned v;
    asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_word(unsigned long long *p, unsigned long long v)
{
    asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ void st_word(unsigned *p, unsigned v)
{
    asm volatile("st.relaxed.gpu.global.b32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// fp32 arithmetic: one word of A and H.  fp64: a word each.  Only finite maps are published, so no word of theirs has all
// bits set.
template <typename A>
struct Words;
template <>
struct Words<float> {
    static constexpr int N = 1;
    using Inc = unsigned;
    unsigned long long w[1];
    static __device__ __forceinline__ void put(unsigned long long *p, float a, float h)
    {
        st_word(p, ((unsigned long long)__float_as_uint(a) << 32) | __float_as_uint(h));
    }
    __device__ __forceinline__ void load(const unsigned long long *p) { w[0] = ld_word(p); }
    __device__ __forceinline__ bool there() const { return (unsigned)(w[0] >> 32) != 0xffffffffu; }
    __device__ __forceinline__ float of(float x) const
    {
        return fma_of(__uint_as_float((unsigned)(w[0] >> 32)), x, __uint_as_float((unsigned)w[0]));
    }
    static __device__ __forceinline__ unsigned inc_bits(float x) { return x == x ? __float_as_uint(x) : 0x7fffffffu; }
    static __device__ __forceinline__ float inc_value(unsigned v) { return __uint_as_float(v); }
    static __device__ __forceinline__ bool inc_there(unsigned v) { return v != 0xffffffffu; }
};
template <>
struct Words<double> {
    static constexpr int N = 2;
    using Inc = unsigned long long;
    static constexpr unsigned long long NONE = ~0ull, QUIET = 0x7ff8000000000000ull;
    unsigned long long w[2];
    static __device__ __forceinline__ unsigned long long bits(double x)
    {
        return x == x ? (unsigned long long)__double_as_longlong(x) : QUIET;
    }
    static __device__ __forceinline__ void put(unsigned long long *p, double a, double h)
    {
        st_word(p, bits(a));
        st_word(p + 1, bits(h));
    }
    __device__ __forceinline__ void load(const unsigned long long *p)
    {
        w[0] = ld_word(p);
        w[1] = ld_word(p + 1);
    }
    __device__ __forceinline__ bool there() const { return w[0] != NONE && w[1] != NONE; }
    __device__ __forceinline__ double of(double x) const
    {
        return fma_of(__longlong_as_double((long long)w[0]), x, __longlong_as_double((long long)w[1]));
    }
    static __device__ __forceinline__ unsigned long long inc_bits(double x) { return bits(x); }
    static __device__ __forceinline__ double inc_value(unsigned long long v) { return __longlong_as_double((long long)v); }
    static __device__ __forceinline__ bool inc_there(unsigned long long v) { return v != NONE; }
};

// One channel's words of the N chunks before `chunk`, nearest first.
template <typename A, int K>
struct Window {
    using Wd = Words<A>;
    typename Wd::Inc v[K];
    Wd m[K];
    __device__ __forceinline__ void load(int last, int64_t n_chan, int64_t ch, const unsigned long long *agg,
                                         const typename Wd::Inc *inc)
    {
        const int64_t at = (int64_t)last * n_chan + ch;
        const typename Wd::Inc *pi = inc + at;
        const unsigned long long *pm = agg + at * Wd::N;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            v[k] = ld_word(pi);
            m[k].load(pm);
            if (last - k > 0) {
                pi -= n_chan;
                pm -= n_chan * Wd::N;
            }
        }
    }
    // Chunk `last - k` is the nearest whose leaving state is there: the state behind all of them in x.
    // 1: yes; 0: a map is missing in front of it; -1: all maps are there and no state
    __device__ __forceinline__ int look(int last, A &x) const
    {
        int found = -1;
        bool open = true;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (open && found < 0) {
                if (last - k >= 0 && Wd::inc_there(v[k])) {
                    found = k;
                    x = Wd::inc_value(v[k]);
                } else
                    open = last - k >= 0 && m[k].there();
            }
        if (found < 0)
            return open ? -1 : 0;
#pragma unroll
        for (int k = K - 2; k >= 0; --k)
            if (k < found)
                x = m[k].of(x);
        return 1;
    }
};

// The state that enters `chunk` at one channel: back to the nearest chunk whose leaving state is there, then
// forward over the maps behind it, one after the other.  FIRST chunks at the first look and while their maps are
// missing, 16 (fp64: 8) further back.
template <typename A, int FIRST>
__device__ __forceinline__ A state_before(int chunk, int64_t n_chan, int64_t ch, const unsigned long long *agg,
                                          const typename Words<A>::Inc *inc)
{
    constexpr int K = 16 / Words<A>::N, LIMIT = 1 << 22;
    A x = A(0);
    int polls = 0, got, last = chunk - 1;
    {
        Window<A, FIRST> near;
        do {
            near.load(last, n_chan, ch, agg, inc);
            got = near.look(last, x);
        } while (got == 0 && ++polls < LIMIT);
        if (got > 0)
            return x;
        last -= FIRST;
    }
    Window<A, K> far;
    while (got <= 0 && polls < LIMIT && last >= 0) {
        far.load(last, n_chan, ch, agg, inc);
        got = far.look(last, x);
        if (got < 0)
            last -= K;
        ++polls;
    }
    if (got <= 0)
        return A(NAN);                                     // gave up
    for (int from = last + 1; from < chunk; from += K) {
        Words<A> m[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            m[k].load(agg + ((int64_t)min(from + k, chunk - 1) * n_chan + ch) * Words<A>::N);
#pragma unroll
        for (int k = 0; k < K; ++k)
            if (from + k < chunk)
                x = m[k].of(x);
    }
    return x;
}

struct TilePlan {
    int tile;                  // -1: no more tiles
    int chunk, cb;
    int lo, hi;                // positions of the tile inside [first, last) row of all sequences
    int first;                 // the sequence that the scan enters at the tile's first position, or -1
    int seg;                   // other borders, or rows outside the sequences, in the tile: use the flags
    int cut;                   // ... such that no state goes through the tile
};

template <typename S, int GATE, bool REV>
struct RecurSmem {
    using P = RecurShape<S, GATE, REV>;
    using A = typename RowType<S>::A;
    static constexpr int NE = P::NIN > P::N1 ? P::NIN - P::N1 : 1;
    // rows of 128 bytes
    uint4 stage0[P::NZ][P::C][8];
    uint4 stage1[P::N1S][P::C][8];
    uint4 stage2[NE][P::NIN > P::N1 ? P::NX : 1][P::NIN > P::N1 ? P::C : 1][8];
    unsigned long long full[P::N1S], late[P::NX];
    // per run and channel (A, H); then the map of the runs in front of it
    A mapA[P::NB][P::NR][P::W], mapH[P::NB][P::NR][P::W];
    A tileA[P::NB][P::W], tileH[P::NB][P::W];      // the tile's map as published
    A enter[P::NB][P::W];                          // the state that enters the tile
    unsigned char fronts[P::NB][P::W];             // how the runs' maps are composed
    int begin[P::NP][P::C], finish[P::NP][P::C];   // sequence the scan enters / leaves at a position, or -1
    TilePlan plan[P::NP];
};

// ------------------------------------------------------------------ the kernel
template <typename S, int GATE, int U, bool REV>
struct Recur {
    using P = RecurShape<S, GATE, REV>;
    using RT = RowType<S>;
    using A = typename RT::A;
    using Sm = RecurSmem<S, GATE, REV>;
    static constexpr int V = P::V, R = P::R, C = P::C, NC = P::NC;
    static constexpr int UNITS = V / U;                    // copies and stores of 16 bytes go in units of U values

    const RecurArgs<S> &g;
    Sm &sm;
    const int tid, warp, lane, l8;
    const int run;                                         // the thread's run of a tile
    const int p0;                                          // its first position
    bool lost = false;                                     // a load did not arrive

    // tid: among the compute threads
    __device__ __forceinline__ Recur(const RecurArgs<S> &g_, Sm &sm_, int tid_)
        : g(g_), sm(sm_), tid(tid_), warp(tid >> 5), lane(threadIdx.x & 31), l8(lane & 7),
          run(tid >> 3), p0(run * R)
    {
    }

    // local channel of element v of the thread
    __device__ __forceinline__ int chan(int v) const { return l8 * V + v; }
    // place of a thread's 16 bytes of channels, and of one channel, in a row of the maps: element v of
    // lane l8 is at (v / Q) 8 Q + l8 Q + v % Q, so that 16-byte accesses of 8 lanes are contiguous
    static constexpr int Q = 16 / (int)sizeof(A);
    static __device__ __forceinline__ int chan_at(int place)
    {
        const int v = place / (8 * Q) * Q + place % Q, l = place / Q % 8;
        return l * V + v;
    }
    __device__ __forceinline__ void put_map(A (&row)[P::W], const A (&x)[V]) const
    {
#pragma unroll
        for (int j = 0; j < V / Q; ++j) {
            uint4 w;
            memcpy(&w, &x[j * Q], 16);
            *reinterpret_cast<uint4 *>(&row[j * 8 * Q + l8 * Q]) = w;
        }
    }
    __device__ __forceinline__ void get_map(const A (&row)[P::W], A (&x)[V]) const
    {
#pragma unroll
        for (int j = 0; j < V / Q; ++j) {
            const uint4 w = *reinterpret_cast<const uint4 *>(&row[j * 8 * Q + l8 * Q]);
            memcpy(&x[j * Q], &w, 16);
        }
    }
    __device__ __forceinline__ int64_t row_of(const TilePlan &pl, int p) const
    {
        const int64_t pos = (int64_t)pl.chunk * C + p;
        return REV ? g.q.n_tokens - 1 - pos : pos;
    }

    __device__ __forceinline__ bool reads(int k) const { return k == 0 || !REV || g.in[k] != nullptr; }

    template <int K>
    __device__ __forceinline__ uint4 *rows_of(int st) const
    {
        return K == 0 ? sm.stage0[st][0] : K == 1 ? sm.stage1[st][0] : sm.stage2[K < 2 ? 0 : K - 2][st][0];
    }
    static constexpr bool BOX = UNITS == 1;                // rows go by tensor copies
    // row of a stage that holds position p: boxes hold rows in memory's order
    static __device__ __forceinline__ int stage_row(int p) { return BOX && REV ? C - 1 - p : p; }

    // One thread starts the copies of a tile's rows of inputs K0 to K1: whole boxes, in which rows outside the sequences
    // are not used and rows outside the array are zeros.
    template <int K0, int K1>
    __device__ __forceinline__ void copy_boxes(const TilePlan &pl, int j, unsigned long long *bar)
    {
        int n = 0;
#pragma unroll
        for (int k = K0; k < K1; ++k)
            n += reads(k) ? 1 : 0;
        mbar_expect(bar, n * C * 128);
        const int x = pl.cb * P::W;
        const int64_t pos = (int64_t)pl.chunk * C;
#pragma unroll
        for (int k = K0; k < K1; ++k) {
            if (!reads(k))
                continue;
            const int y = (int)(REV ? g.q.n_tokens - pos - C : pos) - (REV && k == 2 ? 1 : 0);   // 2: the state before the row
            void *dst = k == 0 ? rows_of<0>(j % P::NZ) : k == 1 ? rows_of<1>(j % P::N1S) : k == 2 ? rows_of<2>(j % P::NX) : rows_of<3>(j % P::NX);
            box_in(dst, &g.map[k], x, y, bar);
        }
    }
    // A warp starts the copies of its 16 rows of input K of a tile, a row (or 128 bytes of two) an instruction.
    template <int K>
    __device__ __forceinline__ void copy_rows(const TilePlan &pl, int st)
    {
        if (!reads(K))
            return;
        constexpr int LANES = P::W / U < 32 ? P::W / U : 32, ROWS = 32 / LANES, TURNS = P::W / U / LANES;
        constexpr int back = REV && K == 2;                // the state before the row
        const int64_t c0 = (int64_t)pl.cb * P::W;
        const int r = lane / LANES, u = lane % LANES * U, first = warp * 16 + r;
        const int64_t t0 = row_of(pl, first) - back;
        const S *src = g.in[K] + t0 * g.ldin[K] + c0 + u;
        S *dst = reinterpret_cast<S *>(rows_of<K>(st) + first * 8) + u;
        const int64_t step = (REV ? -g.ldin[K] : g.ldin[K]) * ROWS;
        const int lo = pl.lo - first, hi = (int)min((int64_t)pl.hi, back ? row_of(pl, 0) : (int64_t)C) - first;
        const int left = (int)min(g.n_chan - c0 - u, (int64_t)P::W);
        if constexpr (U * sizeof(S) >= 4) {
            const int bytes = min(left, U) * (int)sizeof(S);
#pragma unroll
            for (int i = 0; i < 16; i += ROWS, src += step, dst += ROWS * P::W)
                if (i >= lo && i < hi && left > 0)
                    copy_async<U * (int)sizeof(S)>(dst, src, bytes);
        } else {
            constexpr int N = 8;                           // rows in flight
#pragma unroll 1
            for (int i0 = 0; i0 < 16; i0 += N, src += N * step, dst += N * P::W) {
                S x[N][TURNS];
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int k = 0; k < TURNS; ++k)
                        if (i0 + i >= lo && i0 + i < hi && k * LANES < left)
                            x[i][k] = src[i * step + k * LANES];
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int k = 0; k < TURNS; ++k)
                        if (i0 + i >= lo && i0 + i < hi && k * LANES < left)
                            dst[i * P::W + k * LANES] = x[i][k];
            }
        }
    }
    // this thread's copies, or its plain stores, are there
    static __device__ __forceinline__ void arrive(unsigned long long *bar)
    {
        if constexpr (U * sizeof(S) >= 4)
            mbar_arrive_after_copies(bar);
        else
            mbar_arrive(bar);
    }
    // what pass 1 reads of tile j, and what only pass 2 reads: by one thread (BOX) or all compute threads
    __device__ __forceinline__ void load(const TilePlan &pl, int j)
    {
        if (pl.tile < 0)
            return;
        if constexpr (BOX)
            copy_boxes<0, 2>(pl, j, &sm.full[j % P::N1S]);
        else {
            copy_rows<0>(pl, j % P::NZ);
            copy_rows<1>(pl, j % P::N1S);
            arrive(&sm.full[j % P::N1S]);
        }
    }
    __device__ __forceinline__ void load_late(const TilePlan &pl, int j)
    {
        if constexpr (P::NIN > 2) {
            if (pl.tile < 0)
                return;
            if constexpr (BOX)
                copy_boxes<2, P::NIN>(pl, j, &sm.late[j % P::NX]);
            else {
                copy_rows<2>(pl, j % P::NX);
                if constexpr (P::NIN > 3)
                    copy_rows<3>(pl, j % P::NX);
                arrive(&sm.late[j % P::NX]);
            }
        }
    }
    // Wait for what load() started.  A barrier that never ended is marked in `lost`, and from then on the rows of this
    // thread's runs come out as NaN: pass 1 hands over a map that is not finite, pass 2 starts from NaN and spoils the
    // inputs that it reads, so that no first state behind a border makes finite rows of them either.
    __device__ __forceinline__ void loaded(int j)
    {
        lost = !mbar_wait(&sm.full[j % P::N1S], j / P::N1S & 1) || lost;
    }
    __device__ __forceinline__ void loaded_late(int j)
    {
        if constexpr (P::NIN > 2)
            lost = !mbar_wait(&sm.late[j % P::NX], j / P::NX & 1) || lost;
    }
    // The thread's own rows: all bits set, a NaN in every type.
    __device__ __forceinline__ void spoil(int st, int sx)
    {
        const uint4 x = make_uint4(~0u, ~0u, ~0u, ~0u);
#pragma unroll 1
        for (int i = 0; i < R; ++i) {
            const int at = stage_row(p0 + i) * 8 + l8;
            rows_of<1>(st)[at] = x;
            if constexpr (P::NIN > 2)
                rows_of<2>(sx)[at] = x;
        }
    }
    template <int K>
    __device__ __forceinline__ void staged(int st, int i, A (&x)[V]) const
    {
        unpack16(reads(K) ? rows_of<K>(st)[stage_row(p0 + i) * 8 + l8] : make_uint4(0, 0, 0, 0), x, S());
    }
    // One row of states (n_chan fp32 or fp64 values), the thread's channels of it: 16 bytes at a time where that is
    // aligned; zeros where there is none.
    __device__ __forceinline__ bool wide_states(const A *p, int64_t c) const
    {
        return ((uintptr_t)p | (uintptr_t)(g.n_chan * (int64_t)sizeof(A))) % 16 == 0 && c + V <= g.n_chan;
    }
    __device__ __forceinline__ void get_states(const A *p, int s, int64_t c, A (&x)[V]) const
    {
        if (p && wide_states(p, c)) {
            const uint4 *q = reinterpret_cast<const uint4 *>(p + (int64_t)s * g.n_chan + c);
            uint4 r[V / Q];
#pragma unroll
            for (int j = 0; j < V / Q; ++j)
                r[j] = q[j];
            memcpy(x, r, sizeof(r));
        } else
#pragma unroll
            for (int v = 0; v < V; ++v)
                x[v] = p && c + v < g.n_chan ? p[(int64_t)s * g.n_chan + c + v] : A(0);
    }
    __device__ __forceinline__ void put_states(A *p, int s, int64_t c, const A (&x)[V]) const
    {
        if (wide_states(p, c)) {
            uint4 r[V / Q];
            memcpy(r, x, sizeof(r));
#pragma unroll
            for (int j = 0; j < V / Q; ++j)
                reinterpret_cast<uint4 *>(p + (int64_t)s * g.n_chan + c)[j] = r[j];
        } else
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (c + v < g.n_chan)
                    p[(int64_t)s * g.n_chan + c + v] = x[v];
    }

    // What a thread keeps of its coefficients between the passes: a; of a sigmoid the smaller of a and 1 - a, negative
    // (its sign, for 1 - a may be 0) where that is 1 - a, so that both come back with all their digits.
    struct Kept {
        A k[R][V];
    };
    static __device__ __forceinline__ void keep(A (&k)[V], const A (&a)[V], const A (&w)[V])
    {
#pragma unroll
        for (int v = 0; v < V; ++v)
            k[v] = GATE != SLA_GATE_SIGMOID || a[v] <= w[v] ? a[v] : -w[v];
    }
    static __device__ __forceinline__ void kept(const A (&k)[V], A (&a)[V], A (&w)[V])
    {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if constexpr (GATE == SLA_GATE_SIGMOID) {
                const bool other = signbit(k[v]);
                const A rest = add_of(A(1), other ? k[v] : -k[v]);
                a[v] = other ? rest : k[v];
                w[v] = other ? -k[v] : rest;
            } else {
                a[v] = k[v];
                w[v] = A(1);
            }
        }
    }

    // the coefficients and (A, H) of the thread's rows
    template <bool SEG>
    __device__ __forceinline__ void pass1_rows(const TilePlan &pl, int slot, int sz, int st, Kept &kp, A (&ma)[V], A (&mh)[V])
    {
        const int64_t c0 = (int64_t)pl.cb * P::W;
        bool cut = false;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            A z[V], x[V];
            staged<0>(sz, i, z);
            staged<1>(st, i, x);
            const int p = p0 + i;
            int s = -1;
            bool inside = true;
            if constexpr (SEG) {
                inside = p >= pl.lo && p < pl.hi;
                s = inside ? sm.begin[slot][p] : -1;
            }
            A a[V], w[V], y[V];
            gates_of<GATE, sizeof(S) == 2>(z, a, w);
            keep(kp.k[i], a, w);
            if (SEG && s >= 0) {                           // a sequence begins
                get_states(g.enter, s, c0 + l8 * V, mh);
                cut = true;
            }
            const bool first = i == 0 && !(SEG && s >= 0);
            if constexpr (!REV) {
                if constexpr (GATE == SLA_GATE_SIGMOID)
                    vmul(x, w, x);
                if (first)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        mh[v] = x[v];
                else
                    vfma(mh, a, mh, x);
            } else {
                if (first)
                    vmul(mh, a, x);
                else {
                    vadd(y, x, mh);
                    vmul(mh, a, y);
                }
            }
            if (SEG && !inside) {
                vset(mh, A(0));
                cut = true;
            }
            if (i == 0)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    ma[v] = a[v];
            else
                vmul(ma, ma, a);
        }
        // -0 marks a constant map
        if (SEG && cut)
            vset(ma, const_mark<A>());
        else {
            A zero[V];
            vset(zero, A(0));
            vadd(ma, ma, zero);
        }
    }

    __device__ __forceinline__ void pass1(const TilePlan &pl, int slot, int sz, int st, int buf, Kept &kp)
    {
        A ma[V], mh[V];
        if (pl.seg)
            pass1_rows<true>(pl, slot, sz, st, kp, ma, mh);
        else
            pass1_rows<false>(pl, slot, sz, st, kp, ma, mh);
        if (lost)
#pragma unroll
            for (int v = 0; v < V; ++v)
                mh[v] = A(NAN);
        put_map(sm.mapA[buf][run], ma);
        put_map(sm.mapH[buf][run], mh);
    }

    // Row i of the thread's run of output k: to its place in memory, or, where that is not aligned to 16 bytes, to the
    // place of an input that this thread alone has read (input 1 for output 0, input 2 for output 1), from
    // where the warp sends whole rows.
    __device__ __forceinline__ uint4 *out_rows(int k, int st, int sx) const { return k == 0 ? rows_of<1>(st) : rows_of<2>(sx); }
    __device__ __forceinline__ void store(int k, int i, int64_t t, int64_t c0, int st, int sx, const A (&x)[V])
    {
        const uint4 r = pack16(x, S());
        if constexpr (UNITS > 1)
            out_rows(k, st, sx)[(p0 + i) * 8 + l8] = r;
        else {
            S *dst = g.out[k] + t * g.ldout[k] + c0 + l8 * V;
            const int64_t left = g.n_chan - c0 - l8 * V;
            if (left >= V)
                *reinterpret_cast<uint4 *>(dst) = r;
            else {
                S s[V];
                memcpy(s, &r, 16);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (v < left)
                        dst[v] = s[v];
            }
        }
    }
    __device__ __forceinline__ void send_rows(const TilePlan &pl, int st, int sx)
    {
        if constexpr (UNITS > 1) {
            __syncwarp();
            constexpr int N = P::W / 32;                   // channels of a lane, 32 apart
            const int64_t c0 = (int64_t)pl.cb * P::W;
#pragma unroll
            for (int k = 0; k < (REV ? 2 : 1); ++k) {
                if (!g.out[k])
                    continue;
                const S *src = reinterpret_cast<const S *>(out_rows(k, st, sx) + warp * 16 * 8) + lane;
#pragma unroll 4
                for (int r = 0; r < 16; ++r) {
                    const int p = warp * 16 + r;
                    const int64_t t = row_of(pl, p);
                    if ((p >= pl.lo && p < pl.hi) || (g.fill && t >= 0 && t < g.q.n_tokens)) {
                        S *dst = g.out[k] + t * g.ldout[k] + c0 + lane;
#pragma unroll
                        for (int e = 0; e < (N > 0 ? N : 1); ++e)
                            if (lane + 32 * e < P::W && c0 + lane + 32 * e < g.n_chan)
                                dst[32 * e] = src[r * P::W + 32 * e];
                    }
                }
            }
            __syncwarp();                                  // the copies of a later tile into these rows are other lanes'
        }
    }

    template <bool SEG>
    __device__ __forceinline__ void pass2_rows(const TilePlan &pl, int slot, int st, int sx, const Kept &kp, A (&x)[V])
    {
        const int64_t c0 = (int64_t)pl.cb * P::W;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int p = p0 + i;
            const int64_t t = row_of(pl, p);
            int s = -1, f = -1;
            if constexpr (SEG) {
                if (p < pl.lo || p >= pl.hi) {
                    if (g.fill && t >= 0 && t < g.q.n_tokens) {
                        A zero[V];
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            zero[v] = A(0);
                        for (int k = 0; k < (REV ? 2 : 1); ++k)
                            if (g.out[k])
                                store(k, i, t, c0, st, sx, zero);
                    }
                    continue;
                }
                s = sm.begin[slot][p];
                f = sm.finish[slot][p];
            }
            A y[V], a[V], w[V];
            staged<1>(st, i, y);
            kept(kp.k[i], a, w);
            if (SEG && s >= 0)
                get_states(g.enter, s, c0 + l8 * V, x);
            if constexpr (!REV) {
                if constexpr (GATE == SLA_GATE_SIGMOID)
                    vmul(y, w, y);
                vfma(x, a, x, y);
                store(0, i, t, c0, st, sx, x);
            } else {
                A hb[V], lam[V];
                staged<2>(sx, i, hb);
                if (SEG && f >= 0)
                    get_states(g.before, f, c0 + l8 * V, hb);
                vadd(lam, y, x);
                vmul(x, a, lam);
                if constexpr (GATE == SLA_GATE_SIGMOID) {
                    A u[V];
                    staged<3>(sx, i, u);
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        u[v] = -u[v];
                    vadd(hb, hb, u);                       // before - b
                    vmul(lam, w, lam);                     // db
                    vmul(u, x, w);
                    vmul(hb, u, hb);
                } else if constexpr (GATE == SLA_GATE_EXP)
                    vmul(hb, x, hb);
                else
                    vmul(hb, lam, hb);
                if (g.out[0])
                    store(0, i, t, c0, st, sx, lam);
                if (g.out[1])
                    store(1, i, t, c0, st, sx, hb);
            }
            if (SEG && f >= 0 && g.leave)
                put_states(g.leave, f, c0 + l8 * V, x);
        }
    }

    __device__ __forceinline__ void pass2(const TilePlan &pl, int slot, int st, int sx, int buf, const Kept &kp)
    {
        A x[V], a[V], h[V];
        get_map(sm.mapA[buf][run], a);
        get_map(sm.mapH[buf][run], h);
        get_map(sm.enter[buf], x);
#pragma unroll
        for (int v = 0; v < V; ++v)
            x[v] = apply(a[v], x[v], h[v]);
        if (lost) {
            vset(x, A(NAN));
            spoil(st, sx);
        }
        if (pl.seg)
            pass2_rows<true>(pl, slot, st, sx, kp, x);
        else
            pass2_rows<false>(pl, slot, st, sx, kp, x);
        send_rows(pl, st, sx);
    }

    // A channel's runs.  In fp32 a map thread holds them all in registers (their loads then pass at once, and the
    // front maps need no second look); fp64 goes through shared memory twice.
    static constexpr int HELD = sizeof(A) == 4 ? P::NR : 4;
    struct Runs {
        A a[HELD], h[HELD];
    };
    __device__ __forceinline__ void take(int buf, int place, int r0, Runs &q) const
    {
#pragma unroll
        for (int k = 0; k < HELD; ++k) {
            q.a[k] = sm.mapA[buf][r0 + k][place];
            q.h[k] = sm.mapH[buf][r0 + k][place];
        }
    }
    // The tile's (A, H), a constant map's -0 as the factor 0 that it is.  That is right as long as everything is finite, and
    // leaves a result that is not where it is not (infinity times 0): in the order of front_maps(), so that (A, H) is
    // finite only where the maps of all the runs in front are.
    __device__ __forceinline__ void tile_map(int buf, int place, Runs &q, A &ta, A &th) const
    {
        ta = A(1);
        th = A(0);
        for (int r0 = 0; r0 < P::NR; r0 += HELD) {
            if (HELD < P::NR)
                take(buf, place, r0, q);
#pragma unroll
            for (int k = 0; k < HELD; ++k) {
                th = fma_of(q.a[k], th, q.h[k]);
                ta = mul_of(ta, q.a[k]);
            }
        }
    }
    // Every run gets the map of the runs in front of it.  CUT: behind a constant map all are; a product that vanishes
    // is +0, no mark.
    template <bool CUT>
    __device__ __forceinline__ void front_maps(int buf, int place, Runs &q)
    {
        A fa = A(1), fh = A(0);
        bool cut = false;
        for (int r0 = 0; r0 < P::NR; r0 += HELD) {
            if (HELD < P::NR)
                take(buf, place, r0, q);
#pragma unroll
            for (int k = 0; k < HELD; ++k) {
                sm.mapA[buf][r0 + k][place] = CUT && cut ? const_mark<A>() : add_of(fa, A(0));
                sm.mapH[buf][r0 + k][place] = fh;
                fh = fma_of(q.a[k], fh, q.h[k]);
                if (CUT)
                    cut = cut || is_const(q.a[k]);
                fa = mul_of(fa, q.a[k]);
            }
        }
    }
    // The leaving state of a tile with borders, with constant maps looked at: what lies in front of the last one does not
    // count, finite or not.
    static __device__ __noinline__ A last_state(const Sm &sm, int buf, int place)
    {
        A h = A(0);
#pragma unroll 4
        for (int r = 0; r < P::NR; ++r)
            h = apply(sm.mapA[buf][r][place], h, sm.mapH[buf][r][place]);
        return h;
    }
    // A channel of a tile row by row, as pass 2 takes it, from the state x that enters it: where no finite map says what
    // the tile does (a coefficient or an input that is not finite, or a product or sum beyond A's range).  The rows are
    // read from memory again, 16 (fp64: 8) at a time; rare, and out of the way of the others' code.  Returns the
    // state that leaves.  `own`: that it does not depend on x (behind a border or a row outside), or is not finite
    // whatever x is.
    // FRONTS: every run gets the constant map of the state that enters it, which comes from the runs' maps up to the
    // first that is not finite, and again behind a border: those rows keep the bits that they have without it.
    template <bool FRONTS>
    static __device__ __noinline__ A walk(const RecurArgs<S> &g, Sm &sm, int slot, int buf, int place, A x, bool &own)
    {
        constexpr int N = 64 / (int)sizeof(A);
        static_assert(C % N == 0 && N % R == 0, "whole runs");
        const TilePlan pl = sm.plan[slot];
        const int64_t ch = (int64_t)pl.cb * P::W + chan_at(place);
        const A x0 = x;
        A fa = A(1), fh = A(0);
        bool mapped = FRONTS;
        own = false;
#pragma unroll 1
        for (int p0 = 0; p0 < C; p0 += N) {
            if (!pl.seg && isnan(x)) {                     // it stays so: no row is needed
                for (int r = p0 / R; FRONTS && r < P::NR; ++r) {
                    sm.mapA[buf][r][place] = const_mark<A>();
                    sm.mapH[buf][r][place] = x;
                }
                return x;
            }
            A z[N], u[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int64_t pos = (int64_t)pl.chunk * C + p0 + i, t = REV ? g.q.n_tokens - 1 - pos : pos;
                const bool inside = p0 + i >= pl.lo && p0 + i < pl.hi;
                z[i] = inside ? RT::up(g.in[0][t * g.ldin[0] + ch]) : A(0);
                u[i] = inside && (!REV || g.in[1]) ? RT::up(g.in[1][t * g.ldin[1] + ch]) : A(0);
            }
            A a[N], w[N];
            gates_of<GATE, sizeof(S) == 2>(z, a, w);
            if constexpr (!REV && GATE == SLA_GATE_SIGMOID)
                vmul(u, w, u);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int p = p0 + i;
                if (FRONTS && i % R == 0) {
                    A &ra = sm.mapA[buf][p / R][place], &rh = sm.mapH[buf][p / R][place];
                    const A qa = ra, qh = rh;
                    if (mapped)
                        x = apply(fa, x0, fh);
                    ra = const_mark<A>();
                    rh = x;
                    fh = apply(qa, fh, qh);
                    fa = is_const(qa) || is_const(fa) ? const_mark<A>() : add_of(mul_of(fa, qa), A(0));
                    mapped = (mapped || is_const(qa)) && isfinite(fa) && isfinite(fh);
                }
                if (p < pl.lo || p >= pl.hi) {
                    x = A(0);
                    own = true;
                    continue;
                }
                const int s = pl.seg ? sm.begin[slot][p] : -1;
                if (s >= 0) {
                    x = g.enter ? g.enter[(int64_t)s * g.n_chan + ch] : A(0);
                    own = true;
                }
                x = REV ? mul_of(a[i], add_of(u[i], x)) : fma_of(a[i], x, u[i]);
                own = own || !isfinite(u[i]) || isnan(a[i]);
            }
        }
        return mapped ? apply(fa, x0, fh) : x;
    }
    // one channel of a tile: its map, published
    __device__ __forceinline__ void maps(const TilePlan &pl, int buf, int place, Runs &q)
    {
        using Wd = Words<A>;
        const int64_t ch = (int64_t)pl.cb * P::W + chan_at(place);
        A ta, th;
        if (HELD == P::NR)
            take(buf, place, 0, q);
        tile_map(buf, place, q, ta, th);
        A pa = pl.cut ? const_mark<A>() : add_of(ta, A(0));
        int how = pl.cut ? 2 : 1;
        if (!(isfinite(ta) && isfinite(th)) && ch < g.n_chan) {
            how = 0;                                       // there is no map, a state warp goes through the rows
            if (pl.cut)
                th = last_state(sm, buf, place);
            if (!(pl.cut && isfinite(th)))
                pa = A(0);
        }
        sm.fronts[buf][place] = (unsigned char)how;
        sm.tileA[buf][place] = pa;
        sm.tileH[buf][place] = th;
        if (pl.chunk + 1 < g.n_chunks && ch < g.n_chan) {
            const int64_t cell = (int64_t)pl.chunk * g.n_chan + ch;
            if (is_const(pa))
                st_word((typename Wd::Inc *)g.inc + cell, Wd::inc_bits(th));
            else if (how && enters(pl))
                Wd::put(g.agg + cell * Wd::N, pa, th);
        }
    }
    // One channel without a map: a leaving state that does not depend on the entering one is published without waiting for
    // that, so that tiles full of NaN do not wait for one another.
    __device__ __forceinline__ void own_state(const TilePlan &pl, int slot, int buf, int place)
    {
        using Wd = Words<A>;
        if (pl.chunk + 1 == g.n_chunks || is_const(sm.tileA[buf][place]))   // nobody asks, or it is published
            return;
        bool own;
        const A x = walk<false>(g, sm, slot, buf, place, A(0), own);
        if (own)
            st_word((typename Wd::Inc *)g.inc + (int64_t)pl.chunk * g.n_chan + (int64_t)pl.cb * P::W + chan_at(place), Wd::inc_bits(x));
    }

    // whether the tile's own state depends on the chunks before it: not where a border (or a row outside) is at its
    // first position
    __device__ __forceinline__ bool enters(const TilePlan &pl) const
    {
        return pl.chunk > 0 && pl.first < 0 && pl.lo == 0 && pl.hi > 0;
    }
    // one channel of a tile: the state that enters it
    __device__ __forceinline__ A find_state(const TilePlan &pl, int place) const
    {
        const int64_t ch = (int64_t)pl.cb * P::W + chan_at(place);
        if (ch >= g.n_chan)
            return A(0);
        if (pl.first >= 0)
            return g.enter ? g.enter[(int64_t)pl.first * g.n_chan + ch] : A(0);
        if (!enters(pl))
            return A(0);
        // A look waits longer the more words it loads, and loads as many as chunks may be at work (gridDim.x / n_cb): four
        // up to 2.5 of them, eight up to 12, 16 above.  Measured at 2.3 (16384 x 4096 bf16, 64 channel tiles: four 106 us, eight
        // 113, 16 160), 3.7 (32768 x 2560, 40 tiles: eight 132, four 163) and 30 (40000 x 304, 5 tiles: 16 56, eight 60); the
        // borders lie between these.
        const typename Words<A>::Inc *inc = (const typename Words<A>::Inc *)g.inc;
        const int n = (int)gridDim.x;
        if (g.n_cb * 5 >= n * 2)
            return state_before<A, 4>(pl.chunk, g.n_chan, ch, g.agg, inc);
        if (g.n_cb * 12 >= n)
            return state_before<A, 8>(pl.chunk, g.n_chan, ch, g.agg, inc);
        return state_before<A, 16 / Words<A>::N>(pl.chunk, g.n_chan, ch, g.agg, inc);
    }
    // its leaving state, published, and where there is no map the states that enter the runs
    __device__ __forceinline__ void hand_over(const TilePlan &pl, int slot, int buf, int place, A x)
    {
        using Wd = Words<A>;
        const int64_t ch = (int64_t)pl.cb * P::W + chan_at(place);
        const A pa = sm.tileA[buf][place];
        const A th = sm.tileH[buf][place];
        sm.enter[buf][place] = x;
        if (ch >= g.n_chan)
            return;
        bool own = is_const(pa);                              // published by the map warp
        x = sm.fronts[buf][place] ? apply(pa, x, th) : walk<true>(g, sm, slot, buf, place, x, own);
        if (pl.chunk + 1 < g.n_chunks && !own)
            st_word((typename Wd::Inc *)g.inc + (int64_t)pl.chunk * g.n_chan + ch, Wd::inc_bits(x));
    }

    // What the plan warp keeps from tile to tile: the ticket drawn ahead, the first and last row of all sequences, and
    // where the last tile's first sequence was.
    struct PlanState {
        unsigned ticket = 0;
        int64_t lo = 0, hi = 0, hint = 0;
    };
    __device__ __forceinline__ void start(PlanState &ps) const
    {
        if (g.ticket && lane == 0)
            ps.ticket = atomicAdd(g.ticket, 1u);
        if (g.q.n_seq > 0) {
            ps.lo = g.q.at(0);
            ps.hi = max(ps.lo, g.q.at(g.q.n_seq));
        }
    }
    // the plan warp: the next tile, and where sequences begin and end in it
    __device__ __forceinline__ bool plan(int slot, int k, PlanState &ps)
    {
        TilePlan pl;
        const int64_t tiles = (int64_t)g.n_chunks * g.n_cb;
        int64_t tile;
        if (k > 0 && tiles <= gridDim.x)                   // a tile a block
            tile = tiles;
        else if (g.ticket) {
            tile = __shfl_sync(0xffffffffu, ps.ticket + 1u, 0);   // the counter starts at all bits set
            if (lane == 0 && tiles > gridDim.x)
                ps.ticket = atomicAdd(g.ticket, 1u);
        } else
            tile = blockIdx.x + (int64_t)k * gridDim.x;
        if (tile >= tiles) {
            if (lane == 0)
                sm.plan[slot].tile = -1;
            return false;
        }
        pl.tile = (int)tile;
        pl.chunk = (int)(tile / g.n_cb);
        pl.cb = (int)(tile % g.n_cb);
        const int64_t pos0 = (int64_t)pl.chunk * C;
        const int64_t n = g.q.n_tokens;
        const int64_t pos1 = min(n, pos0 + C);
        // the tile's rows in row order
        const int64_t r0 = REV ? n - pos1 : pos0, r1 = REV ? n - pos0 : pos1;
        const int32_t n_seq = g.q.n_seq;
        const int64_t lo = ps.lo, hi = ps.hi;
        const int64_t v0 = min(max(lo, r0), r1), v1 = max(v0, min(hi, r1));
        pl.lo = (int)(REV ? r1 - v1 : v0 - r0);
        pl.hi = (int)(REV ? r1 - v0 : v1 - r0);
        // Offsets are looked at 32 at a time, 31 sequences, from near where the last tile's first one was.  The window
        // is right if nothing in front of it ends behind r0 and something in it does; else the first one
        // that does is searched for, 32 probes at a time.
        int64_t w = n_seq < 32 ? 0 : min(max(ps.hint - (REV ? 24 : 0), (int64_t)0), (int64_t)n_seq - 31);
        auto look = [&] { return w + lane <= n_seq && n_seq > 0 ? g.q.at(w + lane) : INT64_MAX; };
        int64_t off = look();
        const unsigned behind = __ballot_sync(0xffffffffu, lane > 0 && w + lane <= n_seq && off > r0);
        const int64_t off0 = __shfl_sync(0xffffffffu, off, 0);
        if (behind && (w == 0 || off0 <= r0))
            ps.hint = w + __ffs(behind) - 2;
        else if (n_seq >= 32) {
            int64_t s0 = 0, s1 = n_seq;                    // it is in [s0, s1]
            while (s1 - s0 > 32) {
                const int64_t step = (s1 - s0 + 31) / 32;
                const int64_t s = min(s0 + step * (lane + 1) - 1, s1 - 1);
                const unsigned later = __ballot_sync(0xffffffffu, g.q.at(s + 1) > r0);
                const int64_t b0 = s0 + step * (later ? __ffs(later) - 1 : 31);
                s1 = later ? min(s1, b0 + step - 1) : s1;
                s0 = later ? min(b0, s1) : s1;
            }
            ps.hint = w = s0;
            off = look();
        }
        bool seg = pl.lo > 0 || pl.hi < C, cut = seg, cleared = false;
        int first = -1;
        for (;;) {
            const int64_t mine = w + lane, next = __shfl_down_sync(0xffffffffu, off, 1);
            int64_t b = INT64_MAX, e = -1;
            if (lane < 31 && mine < n_seq) {
                b = off;
                e = next - 1;                              // last row
            }
            const bool full = mine < n_seq && e >= b;
            const bool bin = full && b >= r0 && b < r1, ein = full && e >= r0 && e < r1;
            // positions where the scan enters and leaves the sequence
            const int pb = REV ? (int)(r1 - 1 - b) : (int)(b - r0), pe = REV ? (int)(r1 - 1 - e) : (int)(e - r0);
            const int in = REV ? (ein ? pe : -1) : (bin ? pb : -1), leave = REV ? (bin ? pb : -1) : (ein ? pe : -1);
            const unsigned at0 = __ballot_sync(0xffffffffu, in == 0);
            if (at0)
                first = (int)(w + __ffs(at0) - 1);
            cut = __any_sync(0xffffffffu, in > 0) || cut;
            const bool any = cut || __any_sync(0xffffffffu, leave >= 0);
            if ((any || seg) && !cleared) {
                for (int p = lane; p < C; p += 32)
                    sm.begin[slot][p] = sm.finish[slot][p] = -1;
                __syncwarp();
                cleared = seg = true;
            }
            if (in > 0)
                sm.begin[slot][in] = (int)mine;
            if (leave >= 0)
                sm.finish[slot][leave] = (int)mine;
            if (w + 31 >= n_seq || __all_sync(0xffffffffu, b >= r1))
                break;
            w += 31;
            off = look();
        }
        pl.first = first;
        pl.cut = cut;
        pl.seg = seg;
        if (lane == 0)
            sm.plan[slot] = pl;
        return true;
    }
};

// Barriers, each with the warps that arrive and those that wait, one for each of the two tiles at hand: the
// runs' maps are there (compute -> map), the tile's map is there (map -> state), and the front maps, the
// entering states and the plan NS tiles ahead are there (map, state, plan -> compute, plan).
constexpr int BAR_RUNS = 1, BAR_TILE = 3, BAR_ENTER = 5, BAR_START = 7, BAR_FIRST = 8;

template <typename S, int GATE, int U, bool REV>
__global__ void __launch_bounds__(RecurShape<S, GATE, REV>::NT, 1) k_recur(const __grid_constant__ RecurArgs<S> g)
{
    using P = RecurShape<S, GATE, REV>;
    using A = typename RowType<S>::A;
    using K = Recur<S, GATE, U, REV>;
    constexpr int NS = P::NS, NP = P::NP;
    extern __shared__ __align__(128) unsigned char smem_raw[];
    RecurSmem<S, GATE, REV> &sm = *reinterpret_cast<RecurSmem<S, GATE, REV> *>(smem_raw);
    // The warps that the others wait for come first: a scheduler with several warps ready takes the oldest.
    constexpr int STATE = P::NK, PLAN = 2 * P::NK, COMPUTE = PLAN + 32;
    K r(g, sm, (int)threadIdx.x - COMPUTE);
    constexpr int RUNS = P::NC + P::NK, TILE = 2 * P::NK, ENTER = P::NC + 2 * P::NK + 32, START = P::NC + 32;
    auto up = [](int x, int n) { return x + 1 == n ? 0 : x + 1; };
    const int place = threadIdx.x % P::NK;                 // of map and state threads

    if (threadIdx.x >= COMPUTE) {                          // compute warps
        typename K::Kept now, next;
        // while the first plan is made: empty sequences leave with what entered them
        if (g.leave && (g.q.off || g.q.n_tokens == 0))
            for (int64_t s = blockIdx.x; s < g.q.n_seq; s += gridDim.x)
                if (g.q.at(s + 1) <= g.q.at(s))
                    for (int64_t c = r.tid; c < g.n_chan; c += P::NC)
                        g.leave[s * g.n_chan + c] = g.enter ? g.enter[s * g.n_chan + c] : A(0);
        __syncwarp();
        bar_sync(BAR_FIRST, P::NT);                        // plan 0
        if constexpr (!K::BOX) {
            r.load(sm.plan[0], 0);
            r.load_late(sm.plan[0], 0);
            __syncwarp();
        }
        // Plan 1 comes before the map warps hear of tile 0: the state warps look at it once they have tile 0's map.
        bar_sync(BAR_START, START);
        if constexpr (!K::BOX) {
            r.load(sm.plan[1], 1);
            r.load_late(sm.plan[1], 1);
        }
        if (sm.plan[0].tile >= 0) {
            r.loaded(0);
            r.pass1(sm.plan[0], 0, 0, 0, 0, now);
        }
        __syncwarp();
        bar_arrive(BAR_RUNS, RUNS);
        bar_sync(BAR_START, START);                        // plan 2; its stage of input 0 is free after pass 1 of tile 0
        if constexpr (!K::BOX) {
            r.load(sm.plan[2], 2);
            __syncwarp();
        }
        int slot = 0;
        for (int i = 0; sm.plan[slot].tile >= 0; ++i) {
            const int slot1 = up(slot, NP), odd = i & 1;
            if (sm.plan[slot1].tile >= 0) {
                r.loaded(i + 1);
                r.pass1(sm.plan[slot1], slot1, (i + 1) % P::NZ, (i + 1) % P::N1S, odd ^ 1, next);
            }
            __syncwarp();
            bar_arrive(BAR_RUNS + (odd ^ 1), RUNS);        // the first tile there is none of ends the map warps
            bar_sync(BAR_ENTER + odd, ENTER);
            r.loaded_late(i);
            r.pass2(sm.plan[slot], slot, i % P::N1S, i % P::NX, odd, now);
            if constexpr (!K::BOX) {
                const int slot2 = up(slot1, NP);
                r.load(sm.plan[up(slot2, NP)], i + 3);
                r.load_late(sm.plan[slot2], i + 2);
            }
            now = next;
            __syncwarp();
            slot = slot1;
        }
        if constexpr (!K::BOX)
            asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (threadIdx.x < STATE) {                      // map warps
        bar_sync(BAR_FIRST, P::NT);
        for (int slot = 0, odd = 0;; slot = up(slot, NP), odd ^= 1) {
            bar_sync(BAR_RUNS + odd, RUNS);
            const TilePlan &pl = sm.plan[slot];
            if (pl.tile < 0)
                break;
            typename K::Runs q;
            if (place < P::W)
                r.maps(pl, odd, place, q);
            __syncwarp();
            bar_arrive(BAR_TILE + odd, TILE);
            if (place < P::W) {
                const int how = sm.fronts[odd][place];
                if (how == 1)
                    r.template front_maps<false>(odd, place, q);
                else if (how == 2)
                    r.template front_maps<true>(odd, place, q);
                else
                    r.own_state(pl, slot, odd, place);
            }
            __syncwarp();
            bar_arrive(BAR_ENTER + odd, ENTER);
        }
    } else if (threadIdx.x < PLAN) {                       // state warps
        bar_sync(BAR_FIRST, P::NT);
        for (int slot = 0, odd = 0;; slot = up(slot, NP), odd ^= 1) {
            // Plan j is there once tile j - 1's map is: that waits for its runs, and the compute warps hand those over
            // after the barrier that brought plan j (the first for j = 0, the start for 1 and 2, ENTER j - 3).
            const TilePlan &pl = sm.plan[slot];
            if (pl.tile < 0)
                break;
            A x = A(0);
            if (place < P::W)
                x = r.find_state(pl, place);
            __syncwarp();
            bar_sync(BAR_TILE + odd, TILE);
            if (place < P::W)
                r.hand_over(pl, slot, odd, place, x);
            __syncwarp();
            bar_arrive(BAR_ENTER + odd, ENTER);
        }
    } else {                                               // plan warp
        // The compute warps take NS plans before their loop and one in every turn of it, when they are done with the
        // tile before and with pass 1 of the next one: the stages of tile j are free.
        int slot = 0, end = INT32_MAX, odd = 0;
        typename K::PlanState ps;
        r.start(ps);
        if (r.lane == 0) {
            for (int m = 0; m < P::N1S; ++m)
                mbar_init(&sm.full[m], K::BOX ? 1 : P::NC);
            for (int m = 0; m < P::NX; ++m)
                mbar_init(&sm.late[m], K::BOX ? 1 : P::NC);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncwarp();
        for (int j = 0; j < end; ++j) {
            if (end == INT32_MAX) {
                if (!r.plan(slot, j, ps))
                    end = j + NS;
            } else if (r.lane == 0)
                sm.plan[slot].tile = -1;
            __syncwarp();
            if (j == 0)
                bar_sync(BAR_FIRST, P::NT);
            else if (j < NS)
                bar_sync(BAR_START, START);
            else {
                bar_sync(BAR_ENTER + odd, ENTER);
                odd ^= 1;
            }
            if (K::BOX && r.lane == 0) {
                r.load(sm.plan[slot], j);
                if (j >= 2)
                    r.load_late(sm.plan[slot >= 2 ? slot - 2 : slot + NP - 2], j - 2);
            }
            __syncwarp();
            slot = up(slot, NP);
        }
    }
}

// ------------------------------------------------------------------ launch
template <typename S, int GATE, int U, bool REV>
sla_status launch_recur_u(RecurArgs<S> &g, cudaStream_t s)
{
    using P = RecurShape<S, GATE, REV>;
    constexpr size_t smem = sizeof(RecurSmem<S, GATE, REV>);
    static_assert(smem <= 232448, "shared memory of one block");
    static std::atomic<uint64_t> ready{0};                 // devices whose limit is set
    int dev = 0;
    SLA_CUDA_TRY(cudaGetDevice(&dev));
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        SLA_CUDA_TRY(cudaFuncSetAttribute(k_recur<S, GATE, U, REV>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
        if (dev < 64)
            ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    const int64_t tiles = (int64_t)g.n_chunks * g.n_cb;
    const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(tiles, sm_count()));
    k_recur<S, GATE, U, REV><<<grid, P::NT, smem, s>>>(g);
    SLA_CUDA_TRY(cudaGetLastError());
    return SLA_SUCCESS;
}

// cuTensorMapEncodeTiled, looked up once (the library does not link against the driver); NULL if there is none.
using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                                 const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled();

// Rows as boxes of `rows` times 128 bytes.
template <typename S>
bool box_map(CUtensorMap *map, const S *p, int64_t n_tokens, int64_t n_chan, int64_t ld, int rows)
{
    const CUtensorMapDataType type = std::is_same<S, float>::value    ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : std::is_same<S, double>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT64
                                     : std::is_same<S, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                      : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const cuuint64_t dims[2] = {(cuuint64_t)n_chan, (cuuint64_t)n_tokens}, strides[1] = {(cuuint64_t)ld * sizeof(S)};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / sizeof(S)), (cuuint32_t)rows}, each[2] = {1, 1};
    return encode_tiled()(map, type, 2, (void *)p, dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// By alignment: tensor copies where every array's rows are aligned to 16 bytes and every input has a stride (a row
// expanded over the tokens has none); else units of 4 bytes (two of a 16-bit type) or one value.  Copies
// below 4 bytes are not asynchronous.  16384 rows of 1000, 1002 and 1001 bf16: 46, 71 and 128 us; of 1024 and 1001
// fp32: 54 and 91 us; one row of coefficients expanded over 16384 x 4096 bf16 177 us, as many full ones 97.
template <typename S, int GATE, bool REV>
sla_status launch_recur(RecurArgs<S> &g, cudaStream_t s)
{
    using P = RecurShape<S, GATE, REV>;
    uintptr_t bits = 0;
    bool strides = encode_tiled() != nullptr && g.q.n_tokens > 0;
    for (int k = 0; k < 4; ++k)
        if (g.in[k]) {
            bits |= (uintptr_t)g.in[k] | (uintptr_t)(g.ldin[k] * (int64_t)sizeof(S));
            strides = strides && g.ldin[k] > 0 && g.ldin[k] < (int64_t)1 << 36;
        }
    for (int k = 0; k < 2; ++k)
        if (g.out[k])
            bits |= (uintptr_t)g.out[k] | (uintptr_t)(g.ldout[k] * (int64_t)sizeof(S));
    if (bits % 16 == 0 && strides) {
        bool ok = true;
        for (int k = 0; k < 4; ++k)
            if (g.in[k])
                ok = ok && box_map<S>(&g.map[k], g.in[k], g.q.n_tokens, g.n_chan, g.ldin[k], P::C);
        if (ok)
            return launch_recur_u<S, GATE, 16 / (int)sizeof(S), REV>(g, s);
    }
    if constexpr (sizeof(S) == 2)
        if (bits % 4 == 0)
            return launch_recur_u<S, GATE, 2, REV>(g, s);
    return launch_recur_u<S, GATE, 1, REV>(g, s);
}

// Workspace: a line for the ticket, the maps, the leaving states; all bits set before the launch.
template <typename S, int GATE, bool REV>
struct RecurWork {
    using P = RecurShape<S, GATE, REV>;
    using A = typename RowType<S>::A;
    static int64_t chunks(int64_t n_tokens) { return (n_tokens + P::C - 1) / P::C; }
    static size_t per_cell() { return sizeof(unsigned long long) * Words<A>::N + sizeof(A); }
    static size_t bytes(int64_t n_tokens, int64_t n_chan)
    {
        const int64_t n = chunks(n_tokens);
        return n <= 1 ? 0 : 128 + per_cell() * (size_t)n * (size_t)n_chan;
    }
};

// entry points of the two directions (recur_solve.cu, recur_adjoint.cu)
sla_status recur_forward(int32_t dtype, int32_t gate, const void *args, void *work, cudaStream_t s);
sla_status recur_backward(int32_t dtype, int32_t gate, const void *args, void *work, cudaStream_t s);

template <class F>
static inline sla_status with_gate(int32_t gate, F f)
{
    switch (gate) {
    case SLA_GATE_VALUE: return f(std::integral_constant<int, SLA_GATE_VALUE>());
    case SLA_GATE_EXP: return f(std::integral_constant<int, SLA_GATE_EXP>());
    default: return f(std::integral_constant<int, SLA_GATE_SIGMOID>());
    }
}

template <typename S, bool REV>
sla_status run_recur(int32_t gate, RecurArgs<S> g, void *work, cudaStream_t s)
{
    using A = typename RowType<S>::A;
    return with_gate(gate, [&](auto tag) -> sla_status {
        constexpr int GATE = decltype(tag)::value;
        using Wk = RecurWork<S, GATE, REV>;
        const int64_t chunks = Wk::chunks(g.q.n_tokens), cb = (g.n_chan + RecurShape<S, GATE, REV>::W - 1) / RecurShape<S, GATE, REV>::W;
        if (chunks * cb > INT32_MAX)
            return fail(SLA_ERR_UNSUPPORTED, "more than 2^31 tiles of rows and channels");
        g.n_chunks = (int)chunks;
        g.n_cb = (int)cb;
        g.ticket = nullptr;
        g.agg = nullptr;
        g.inc = nullptr;
        const size_t need = Wk::bytes(g.q.n_tokens, g.n_chan);
        if (need) {
            SLA_CUDA_TRY(cudaMemsetAsync(work, 0xff, need, s));
            g.ticket = (unsigned *)work;
            g.agg = (unsigned long long *)((char *)work + 128);
            g.inc = (char *)g.agg + sizeof(unsigned long long) * Words<A>::N * (size_t)chunks * (size_t)g.n_chan;
        }
        return launch_recur<S, GATE, REV>(g, s);
    });
}

}  // namespace sla
