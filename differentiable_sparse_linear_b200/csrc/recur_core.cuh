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
// One block runs four kinds of work at the same time, tile i being the oldest:
//   loads       each thread copies its own rows of tile i + NS into its own place in shared memory
//               (cp.async), so staging needs no barrier;
//   pass 1      tile i + 1: each thread's (A, H), left in shared memory;
//   scan warps  tile i + 1, four threads a channel, each over a quarter of the runs in order: the tile's (A, H),
//               published for later chunks; the state that enters it, from the published results of
//               earlier chunks; the state that enters every run;
//   pass 2      tile i: every row from the state that enters it, in the order of the formula, and the stores.
// A plan warp takes the tickets and finds the sequence borders inside a tile, NS tiles ahead.  So each
// input is read once and the wait on earlier chunks passes while other tiles are worked on.
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
// A sequence border inside a run makes its map constant.  Such a map is marked by A = -0 (products are
// normalised to +0), because 0 * x would carry a NaN or an infinity across the border.  Where the entering state is
// exactly 0, A is not used, so that a product of large coefficients that overflowed does no harm to rows
// of zeros.
#pragma once

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
    static constexpr int R = 4;
    // Warps and stages by shared memory (three stages, so that a load has a tile's time to arrive)
    static constexpr int NW = !REV ? 12 : NIN == 3 ? 10 : 7;
    static constexpr int NS = 3;
    static constexpr int NP = NS + 1;                      // plan slots
    static constexpr int NR = NW * 4;                      // runs
    static constexpr int C = NR * R;
    static constexpr int NC = NW * 32;                     // compute threads
    static constexpr int RQ = NR / 4;                      // runs of a quarter of the tile
    static constexpr int NSCAN = W * 4;                    // scan threads: four a channel, a quarter each
    static constexpr int NT = NC + NSCAN + 32;
};

struct TilePlan {
    int tile;                  // -1: no more tiles
    int chunk, cb;
    int lo, hi;                // positions of the tile inside [first, last) row of all sequences
    int seg;                   // borders or rows outside the sequences in the tile: use the flags
};

template <typename S, int GATE, bool REV>
struct RecurSmem {
    using P = RecurShape<S, GATE, REV>;
    using A = typename RowType<S>::A;
    uint4 stage[P::NS][P::NIN][P::R][P::NC];
    // per run and channel (A, H); the scan leaves the state that enters the run in H's place
    A mapA[2][P::NR][P::W], mapH[2][P::NR][P::W];
    int begin[P::NP][P::C], finish[P::NP][P::C];   // sequence the scan enters / leaves at a position, or -1
    TilePlan plan[P::NP];
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

// ------------------------------------------------------------------ affine maps
__device__ __forceinline__ bool is_const(float a) { return __float_as_uint(a) == 0x80000000u; }
__device__ __forceinline__ bool is_const(double a) { return (unsigned long long)__double_as_longlong(a) == 0x8000000000000000ull; }
template <typename A>
__device__ __forceinline__ A const_mark() { return A(-0.0); }
// x -> A x + H at x; at x = 0 without A, which may have overflowed.
template <typename A, typename B>
__device__ __forceinline__ B apply(A a, B x, B h)
{
    return (is_const(a) || x == B(0)) ? h : fma_of(B(a), x, h);
}
// The product of a later a2 and an earlier a1.
template <typename A>
__device__ __forceinline__ A product(A a2, A a1)
{
    return (is_const(a1) || is_const(a2)) ? const_mark<A>() : a2 * a1 + A(0);
}
// apply() with an A wider than fp32's range (published maps): the fp64 product, rounded once with the sum
__device__ __forceinline__ float apply_wide(double a, float x, float h)
{
    return (is_const(a) || x == 0.0f) ? h : (float)__fma_rn(a, (double)x, (double)h);
}
__device__ __forceinline__ double apply_wide(double a, double x, double h) { return apply(a, x, h); }

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

// fp32 arithmetic: A's upper 32 bits as fp64 (its range; 2^-21 relative, once per chunk) and H in one word.
// fp64: a word each.
template <typename A>
struct Words;
template <>
struct Words<float> {
    static constexpr int N = 1;
    using Inc = unsigned;
    unsigned long long w[1];
    // A as it is published: every user of the map, its own chunk included, applies this one
    static __device__ __forceinline__ double round_a(double a)
    {
        if (!(a == a))
            return __hiloint2double(0x7ff80000, 0);
        return __longlong_as_double((__double_as_longlong(a) + 0x80000000ll) & ~0xffffffffll);
    }
    static __device__ __forceinline__ void put(unsigned long long *p, double a, float h)
    {
        st_word(p, ((unsigned long long)(unsigned)__double2hiint(a) << 32) | __float_as_uint(h));
    }
    __device__ __forceinline__ void load(const unsigned long long *p) { w[0] = ld_word(p); }
    __device__ __forceinline__ bool there() const { return (unsigned)(w[0] >> 32) != 0xffffffffu; }
    __device__ __forceinline__ double a() const { return __hiloint2double((int)(w[0] >> 32), 0); }
    __device__ __forceinline__ float h() const { return __uint_as_float((unsigned)w[0]); }
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
    static __device__ __forceinline__ double round_a(double a) { return a; }
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
    __device__ __forceinline__ double a() const { return __longlong_as_double((long long)w[0]); }
    __device__ __forceinline__ double h() const { return __longlong_as_double((long long)w[1]); }
    static __device__ __forceinline__ unsigned long long inc_bits(double x) { return bits(x); }
    static __device__ __forceinline__ double inc_value(unsigned long long v) { return __longlong_as_double((long long)v); }
    static __device__ __forceinline__ bool inc_there(unsigned long long v) { return v != NONE; }
};

// The state that enters `chunk` at one channel, by the four lanes l, l + 8, l + 16, l + 24 of a warp: back to the
// nearest chunk whose leaving state is there (4 K chunks a round trip, K a lane), then forward over the
// maps behind it, one after the other.  All lanes of the warp call it; `want` is false where no state is needed.
template <typename A>
__device__ __forceinline__ A state_before(int chunk, int64_t n_chan, int64_t ch, bool want, int lane,
                                          const unsigned long long *agg, const typename Words<A>::Inc *inc)
{
    using Wd = Words<A>;
    constexpr int K = 4, OPEN = 1 << 20;
    const unsigned all = 0xffffffffu;
    const int q = lane >> 3, l8 = lane & 7;
    bool done = !want, gave_up = false;
    A x = A(0);
    int last = chunk - 1, from = chunk;
    for (int polls = 0;; ++polls) {
        typename Wd::Inc v[K];
        Wd m[K];
        int mine = OPEN;               // 2 * (distance) of the nearest leaving state, + 1 if a map is missing first
        if (!done) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int64_t at = (int64_t)max(last - q * K - k, 0) * n_chan + ch;
                v[k] = ld_word(inc + at);
                m[k].load(agg + at * Wd::N);
            }
#pragma unroll
            for (int k = K - 1; k >= 0; --k)
                if (last - q * K - k >= 0) {
                    if (Wd::inc_there(v[k]))
                        mine = 2 * (q * K + k);
                    else if (!m[k].there())
                        mine = 2 * (q * K + k) + 1;
                }
        }
        mine = min(mine, __shfl_xor_sync(all, mine, 8));
        mine = min(mine, __shfl_xor_sync(all, mine, 16));
        const bool found = !done && mine < OPEN && !(mine & 1);
        if (__any_sync(all, found)) {
            const int fq = mine / 2 / K, fk = mine / 2 % K;
            A y = A(0);
#pragma unroll
            for (int k = 0; k < K; ++k)
                if (found && q == fq && k == fk)
                    y = Wd::inc_value(v[k]);
#pragma unroll
            for (int s = 3; s >= 0; --s) {
                if (found && q == s && s <= fq) {
#pragma unroll
                    for (int k = K - 1; k >= 0; --k)
                        if (s < fq || k < fk)
                            y = apply_wide(m[k].a(), y, m[k].h());
                }
                const A o = __shfl_sync(all, y, s * 8 + l8);
                if (q < s && s <= fq)
                    y = o;
            }
            y = __shfl_sync(all, y, l8);
            if (found) {
                x = y;
                from = last + 1;
                done = true;
            }
        }
        if (!done && mine == OPEN && last - 4 * K >= 0)
            last -= 4 * K;
        if (!__any_sync(all, !done))
            break;
        if (polls >= 1 << 22) {
            gave_up = !done;
            break;
        }
    }
    // the maps that were passed on the way back
    while (__any_sync(all, from < chunk)) {
        Wd m[K];
#pragma unroll
        for (int k = 0; k < K; ++k)
            m[k].load(agg + ((int64_t)min(from + q * K + k, chunk - 1) * n_chan + ch) * Wd::N);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (q == s) {
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (from + q * K + k < chunk)
                        x = apply_wide(m[k].a(), x, m[k].h());
            }
            x = __shfl_sync(all, x, s * 8 + l8);
        }
        from += 4 * K;
    }
    return gave_up ? A(NAN) : x;
}

// ------------------------------------------------------------------ the kernel
template <typename S, int GATE, int U, bool REV>
struct Recur {
    using P = RecurShape<S, GATE, REV>;
    using RT = RowType<S>;
    using A = typename RT::A;
    using Sm = RecurSmem<S, GATE, REV>;
    static constexpr int V = P::V, R = P::R, C = P::C, NC = P::NC;
    static constexpr int UNITS = V / U;                    // a thread's channels: UNITS groups of U contiguous ones

    const RecurArgs<S> &g;
    Sm &sm;
    const int tid, warp, lane, l8;
    const int run;                                         // the thread's run of a tile
    const int p0;                                          // its first position

    __device__ __forceinline__ Recur(const RecurArgs<S> &g_, Sm &sm_)
        : g(g_), sm(sm_), tid(threadIdx.x), warp(tid >> 5), lane(tid & 31), l8(lane & 7),
          run(tid >> 3), p0(run * R)
    {
    }

    // local channel of element v of the thread
    __device__ __forceinline__ int chan(int v) const { return ((v / U) * 8 + l8) * U + v % U; }
    // Place of a thread's 16 bytes of channels, and of one channel, in a row of the maps: element v of
    // lane l8 is at (v / Q) 8 Q + l8 Q + v % Q, so that 16-byte accesses of 8 lanes are contiguous; a quarter's
    // rows are turned by 8 places, so that a scan warp (8 places of four quarters) meets no bank twice.
    static constexpr int Q = 16 / (int)sizeof(A);
    static __device__ __forceinline__ int turn(int quarter) { return (quarter * 8) & (P::W - 1); }
    static __device__ __forceinline__ int chan_at(int place)
    {
        const int v = place / (8 * Q) * Q + place % Q, l = place / Q % 8;
        return ((v / U) * 8 + l) * U + v % U;
    }
    __device__ __forceinline__ void put_map(A (*m)[P::W], const A (&x)[V]) const
    {
#pragma unroll
        for (int j = 0; j < V / Q; ++j) {
            uint4 w;
            memcpy(&w, &x[j * Q], 16);
            *reinterpret_cast<uint4 *>(&m[run][(j * 8 * Q + l8 * Q) ^ turn(run / P::RQ)]) = w;
        }
    }
    __device__ __forceinline__ void get_map(A (*m)[P::W], A (&x)[V]) const
    {
#pragma unroll
        for (int j = 0; j < V / Q; ++j) {
            const uint4 w = *reinterpret_cast<const uint4 *>(&m[run][(j * 8 * Q + l8 * Q) ^ turn(run / P::RQ)]);
            memcpy(&x[j * Q], &w, 16);
        }
    }
    __device__ __forceinline__ int64_t row_of(const TilePlan &pl, int p) const
    {
        const int64_t pos = (int64_t)pl.chunk * C + p;
        return REV ? g.q.n_tokens - 1 - pos : pos;
    }

    __device__ __forceinline__ bool reads(int k) const { return g.in[k] != nullptr; }

    // start the copies of the thread's rows of a tile
    template <bool SEG>
    __device__ __forceinline__ void load_rows(const TilePlan &pl, int st)
    {
        const int64_t c0 = (int64_t)pl.cb * P::W;
        const int64_t t0 = row_of(pl, p0);
#pragma unroll
        for (int k = 0; k < P::NIN; ++k) {
            if (!reads(k))
                continue;
            const int back = REV && k == 2;                // the state before the row
            const S *src = g.in[k] + (t0 - back) * g.ldin[k] + c0;
            const int64_t step = REV ? -g.ldin[k] : g.ldin[k];
#pragma unroll
            for (int i = 0; i < R; ++i, src += step) {
                const int p = p0 + i;
                if (SEG && (p < pl.lo || p >= pl.hi))
                    continue;
                if (back && t0 - i <= 0)
                    continue;
                S *dst = reinterpret_cast<S *>(&sm.stage[st][k][i][tid]);
#pragma unroll
                for (int j = 0; j < UNITS; ++j) {
                    const int c = chan(j * U);
                    const int64_t left = g.n_chan - c0 - c;
                    if (left <= 0)
                        continue;
                    if constexpr (U * sizeof(S) >= 4)
                        copy_async<U * (int)sizeof(S)>(dst + j * U, src + c, (int)min(left, (int64_t)U) * (int)sizeof(S));
                    else
                        dst[j] = src[c];
                }
            }
        }
    }
    __device__ __forceinline__ void load(const TilePlan &pl, int st)
    {
        if (pl.tile >= 0) {
            if (pl.seg)
                load_rows<true>(pl, st);
            else
                load_rows<false>(pl, st);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    __device__ __forceinline__ void staged(int st, int k, int i, A (&x)[V]) const
    {
        const uint4 r = reads(k) ? sm.stage[st][k][i][tid] : make_uint4(0, 0, 0, 0);
        unpack16(r, x, S());
    }
    __device__ __forceinline__ A enter_of(int s, int64_t ch) const
    {
        return g.enter && ch < g.n_chan ? g.enter[(int64_t)s * g.n_chan + ch] : A(0);
    }

    // (A, H) of the thread's rows
    template <bool SEG>
    __device__ __forceinline__ void pass1_rows(const TilePlan &pl, int slot, int st, A (&ma)[V], A (&mh)[V])
    {
        const int64_t c0 = (int64_t)pl.cb * P::W;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            A z[V], x[V];
            staged(st, 0, i, z);
            staged(st, 1, i, x);
            const int p = p0 + i;
            int s = -1;
            bool inside = true;
            if constexpr (SEG) {
                inside = p >= pl.lo && p < pl.hi;
                s = inside ? sm.begin[slot][p] : -1;
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                A a, w;
                gate_of<GATE, sizeof(S) == 2>(z[v], a, w);
                A h;
                if constexpr (!REV) {
                    const A u = w * x[v];
                    h = i == 0 ? u : fma_of(a, mh[v], u);
                    if (SEG && s >= 0)
                        h = g.enter ? fma_of(a, enter_of(s, c0 + chan(v)), u) : u;
                } else {
                    A y = i == 0 ? x[v] : add_of(x[v], mh[v]);
                    if (SEG && s >= 0)
                        y = add_of(x[v], enter_of(s, c0 + chan(v)));
                    h = mul_of(a, y);
                }
                if constexpr (SEG) {
                    A m = i == 0 ? a + A(0) : product(a, ma[v]);
                    if (s >= 0)
                        m = const_mark<A>();
                    if (!inside) {
                        m = const_mark<A>();
                        h = A(0);
                    }
                    ma[v] = m;
                } else
                    ma[v] = i == 0 ? a : i == R - 1 ? ma[v] * a + A(0) : ma[v] * a;
                mh[v] = h;
            }
        }
    }

    __device__ __forceinline__ void pass1(const TilePlan &pl, int slot, int st, int buf)
    {
        A ma[V], mh[V];
        if (pl.seg)
            pass1_rows<true>(pl, slot, st, ma, mh);
        else
            pass1_rows<false>(pl, slot, st, ma, mh);
        put_map(sm.mapA[buf], ma);
        put_map(sm.mapH[buf], mh);
    }

    __device__ __forceinline__ void store(int k, int64_t t, int64_t c0, const A (&x)[V])
    {
        S *dst = g.out[k] + t * g.ldout[k] + c0;
        const uint4 r = pack16(x, S());
        S s[V];
        memcpy(s, &r, 16);
#pragma unroll
        for (int j = 0; j < UNITS; ++j) {
            const int c = chan(j * U);
            const int64_t left = g.n_chan - c0 - c;
            if (left >= U) {
                if constexpr (UNITS == 1)
                    *reinterpret_cast<uint4 *>(dst + c) = r;
                else if constexpr (U == 1)
                    dst[c] = s[j];
                else {
                    unsigned w;
                    memcpy(&w, s + j * U, 4);
                    *reinterpret_cast<unsigned *>(dst + c) = w;
                }
            } else if constexpr (U > 1) {
#pragma unroll
                for (int e = 0; e < U; ++e)
                    if (e < left)
                        dst[c + e] = s[j * U + e];
            }
        }
    }

    template <bool SEG>
    __device__ __forceinline__ void pass2_rows(const TilePlan &pl, int slot, int st, A (&x)[V])
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
                                store(k, t, c0, zero);
                    }
                    continue;
                }
                s = sm.begin[slot][p];
                f = sm.finish[slot][p];
            }
            A z[V], y[V];
            staged(st, 0, i, z);
            staged(st, 1, i, y);
            if constexpr (!REV) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    A a, w;
                    gate_of<GATE, sizeof(S) == 2>(z[v], a, w);
                    const A u = w * y[v];
                    if (SEG && s >= 0)
                        x[v] = g.enter ? fma_of(a, enter_of(s, c0 + chan(v)), u) : u;
                    else
                        x[v] = fma_of(a, x[v], u);
                }
                store(0, t, c0, x);
            } else {
                A hb[V], u[V], db[V], dz[V];
                staged(st, 2, i, hb);
                if constexpr (GATE == SLA_GATE_SIGMOID)
                    staged(st, 3, i, u);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    A a, w;
                    gate_of<GATE, sizeof(S) == 2>(z[v], a, w);
                    const A lam = add_of(y[v], SEG && s >= 0 ? enter_of(s, c0 + chan(v)) : x[v]);
                    A hp = hb[v];
                    if (SEG && f >= 0) {
                        const int64_t ch = c0 + chan(v);
                        hp = g.before && ch < g.n_chan ? g.before[(int64_t)f * g.n_chan + ch] : A(0);
                    }
                    x[v] = mul_of(a, lam);
                    db[v] = w * lam;
                    if constexpr (GATE == SLA_GATE_VALUE)
                        dz[v] = lam * hp;
                    else if constexpr (GATE == SLA_GATE_EXP)
                        dz[v] = x[v] * hp;
                    else
                        dz[v] = x[v] * w * (hp - u[v]);
                }
                if (g.out[0])
                    store(0, t, c0, db);
                if (g.out[1])
                    store(1, t, c0, dz);
            }
            if (SEG && f >= 0 && g.leave) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int64_t ch = c0 + chan(v);
                    if (ch < g.n_chan)
                        g.leave[(int64_t)f * g.n_chan + ch] = x[v];
                }
            }
        }
    }

    __device__ __forceinline__ void pass2(const TilePlan &pl, int slot, int st, int buf)
    {
        A x[V];
        get_map(sm.mapH[buf], x);
        if (pl.seg)
            pass2_rows<true>(pl, slot, st, x);
        else
            pass2_rows<false>(pl, slot, st, x);
    }

    // (A, H) of consecutive runs.  Without borders in the tile no map is constant, and the guard against
    // an overflowed A times 0 is needed only if a NaN comes out.  The products of four runs stay in fp32
    // (16 coefficients), longer ones are taken in fp64.
    template <bool GUARD>
    static __device__ __forceinline__ void compose(const A (&a)[P::RQ], const A (&h)[P::RQ], double &ta, A &th)
    {
        th = h[0];
#pragma unroll
        for (int k = 1; k < P::RQ; ++k)
            th = GUARD ? apply(a[k], th, h[k]) : fma_of(a[k], th, h[k]);
#pragma unroll
        for (int k = 0; k < P::RQ; k += 4) {
            A m = a[k];
#pragma unroll
            for (int e = 1; e < 4; ++e)
                if (k + e < P::RQ)
                    m = GUARD ? product(a[k + e], m) : a[k + e] * m;
            if constexpr (GUARD)
                ta = k ? product((double)m, ta) : (double)m;
            else
                ta = k ? (double)m * ta : (double)m;
        }
        if constexpr (!GUARD)
            ta += 0.0;                                     // -0 marks a constant map
    }
    // Every run gets the state that enters it.
    template <bool GUARD>
    __device__ __forceinline__ void enter_runs(int buf, int r0, int at, const A (&a)[P::RQ], const A (&h)[P::RQ], A x)
    {
#pragma unroll
        for (int k = 0; k < P::RQ; ++k) {
            sm.mapH[buf][r0 + k][at] = x;
            x = GUARD ? apply(a[k], x, h[k]) : fma_of(a[k], x, h[k]);
        }
    }

    // 8 channels of a tile by a warp: publish, find the state that enters, hand it to the runs
    __device__ __forceinline__ void scan(const TilePlan &pl, int slot, int buf, int sw)
    {
        using Wd = Words<A>;
        const unsigned all = 0xffffffffu;
        const int q = lane >> 3, place = sw * 8 + l8, at = place ^ turn(q), r0 = q * P::RQ;
        const int64_t ch = (int64_t)pl.cb * P::W + chan_at(place);
        const bool real = ch < g.n_chan;
        A a[P::RQ], h[P::RQ], th, x = A(0);
        double ta;
#pragma unroll
        for (int k = 0; k < P::RQ; ++k) {
            a[k] = sm.mapA[buf][r0 + k][at];
            h[k] = sm.mapH[buf][r0 + k][at];
        }
        if (pl.seg)
            compose<true>(a, h, ta, th);
        else {
            compose<false>(a, h, ta, th);
            if (!(th == th))
                compose<true>(a, h, ta, th);
        }
        const bool plain = !pl.seg && __all_sync(all, isfinite(ta) || !real);
        // over the quarters; (pa, ph): the quarters in front
#pragma unroll
        for (int d = 8; d < 32; d *= 2) {
            const double oa = __shfl_up_sync(all, ta, d);
            const A oh = __shfl_up_sync(all, th, d);
            if (lane >= d) {
                th = apply_wide(ta, oh, th);
                ta = product(ta, oa);
            }
        }
        const double pa = __shfl_up_sync(all, ta, 8);
        const A ph = __shfl_up_sync(all, th, 8);
        if (g.n_chunks > 1) {
            ta = Wd::round_a(__shfl_sync(all, ta, 24 + l8));
            th = __shfl_sync(all, th, 24 + l8);
            const int64_t cell = (int64_t)pl.chunk * g.n_chan + ch;
            typename Wd::Inc *inc = (typename Wd::Inc *)g.inc;
            const bool first = pl.chunk == 0, fixed = first || is_const(ta);
            const bool publish = q == 3 && real && pl.chunk + 1 < g.n_chunks;
            if (publish) {
                if (fixed)
                    st_word(inc + cell, Wd::inc_bits(th));
                else
                    Wd::put(g.agg + cell * Wd::N, ta, th);
            }
            // a border (or a row outside) at the first position: nothing enters
            if (!first && !(pl.seg && (pl.lo > 0 || pl.hi == 0 || sm.begin[slot][0] >= 0))) {
                x = state_before<A>(pl.chunk, g.n_chan, ch, real, lane, g.agg, inc);
                if (publish && !fixed)
                    st_word(inc + cell, Wd::inc_bits(apply_wide(ta, x, th)));
            }
        }
        if (q > 0)
            x = apply_wide(pa, x, ph);
        // The guard is needed with constant maps, and where a run's A overflowed, which leaves its quarter's
        // not finite.
        if (plain)
            enter_runs<false>(buf, r0, at, a, h, x);
        else
            enter_runs<true>(buf, r0, at, a, h, x);
    }

    // the plan warp: the next tile, and where sequences begin and end in it
    __device__ __forceinline__ bool plan(int slot, int k)
    {
        TilePlan pl;
        const int64_t tiles = (int64_t)g.n_chunks * g.n_cb;
        int64_t tile;
        if (g.ticket) {
            unsigned v = 0;
            if (lane == 0)
                v = atomicAdd(g.ticket, 1u) + 1u;          // the counter starts at all bits set
            tile = __shfl_sync(0xffffffffu, v, 0);
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
        const int64_t lo = g.q.n_seq > 0 ? g.q.at(0) : 0, hi = g.q.n_seq > 0 ? max(lo, g.q.at(g.q.n_seq)) : 0;
        const int64_t v0 = min(max(lo, r0), r1), v1 = max(v0, min(hi, r1));
        pl.lo = (int)(REV ? r1 - v1 : v0 - r0);
        pl.hi = (int)(REV ? r1 - v0 : v1 - r0);
        // the first sequence that ends behind r0: of 32 probes at a time
        int64_t s0 = 0, s1 = g.q.n_seq;                    // it is in [s0, s1]
        while (s1 - s0 > 32) {
            const int64_t step = (s1 - s0 + 31) / 32;
            const int64_t s = min(s0 + step * (lane + 1) - 1, s1 - 1);
            const unsigned behind = __ballot_sync(0xffffffffu, g.q.at(s + 1) > r0);
            const int k0 = behind ? __ffs(behind) - 1 : 31;
            const int64_t b0 = s0 + step * k0;
            s1 = behind ? min(s1, b0 + step - 1) : s1;
            s0 = min(b0, s1);
            if (!behind)
                s0 = s1;
        }
        bool seg = pl.lo > 0 || pl.hi < C, cleared = false;
        for (int64_t s = s0;; s += 32) {
            const int64_t mine = s + lane;
            int64_t b = INT64_MAX, e = -1;
            if (mine < g.q.n_seq) {
                b = g.q.at(mine);
                e = g.q.at(mine + 1) - 1;                  // last row
            }
            const bool full = e >= b && mine < g.q.n_seq;
            const bool bin = full && b >= r0 && b < r1, ein = full && e >= r0 && e < r1;
            const bool any = __any_sync(0xffffffffu, bin || ein);
            if ((any || seg) && !cleared) {
                for (int p = lane; p < C; p += 32)
                    sm.begin[slot][p] = sm.finish[slot][p] = -1;
                __syncwarp();
                cleared = seg = true;
            }
            if (bin)
                (REV ? sm.finish : sm.begin)[slot][REV ? (int)(r1 - 1 - b) : (int)(b - r0)] = (int)mine;
            if (ein)
                (REV ? sm.begin : sm.finish)[slot][REV ? (int)(r1 - 1 - e) : (int)(e - r0)] = (int)mine;
            const int64_t next = s + 32;
            if (next >= g.q.n_seq || __all_sync(0xffffffffu, b >= r1))
                break;
        }
        pl.seg = seg;
        if (lane == 0)
            sm.plan[slot] = pl;
        return true;
    }
};

constexpr int BAR_P1 = 1, BAR_P2 = 3, BAR_PLAN = 5;

template <typename S, int GATE, int U, bool REV>
__global__ void __launch_bounds__(RecurShape<S, GATE, REV>::NT, 1) k_recur(const __grid_constant__ RecurArgs<S> g)
{
    using P = RecurShape<S, GATE, REV>;
    using A = typename RowType<S>::A;
    constexpr int NS = P::NS, NP = P::NP;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    RecurSmem<S, GATE, REV> &sm = *reinterpret_cast<RecurSmem<S, GATE, REV> *>(smem_raw);
    Recur<S, GATE, U, REV> r(g, sm);

    if (r.tid < P::NC) {                                   // compute warps
        for (int j = 0; j < NS; ++j) {
            bar_sync(BAR_PLAN, P::NC + 32);
            r.load(sm.plan[j], j);
            __syncwarp();
        }
        asm volatile("cp.async.wait_group %0;" ::"n"(NS - 1) : "memory");
        if (sm.plan[0].tile >= 0)
            r.pass1(sm.plan[0], 0, 0, 0);
        __syncwarp();
        bar_arrive(BAR_P1, P::NC + P::NSCAN);
        int st = 0, slot = 0, buf = 0;
        while (sm.plan[slot].tile >= 0) {
            const int st1 = st + 1 == NS ? 0 : st + 1, slot1 = slot + 1 == NP ? 0 : slot + 1;
            asm volatile("cp.async.wait_group %0;" ::"n"(NS - 2) : "memory");
            if (sm.plan[slot1].tile >= 0)
                r.pass1(sm.plan[slot1], slot1, st1, buf ^ 1);
            __syncwarp();
            bar_arrive(BAR_P1 + (buf ^ 1), P::NC + P::NSCAN);
            bar_sync(BAR_P2 + buf, P::NC + P::NSCAN);
            r.pass2(sm.plan[slot], slot, st, buf);
            __syncwarp();
            bar_sync(BAR_PLAN, P::NC + 32);
            const int ahead = slot + NS >= NP ? slot + NS - NP : slot + NS;
            r.load(sm.plan[ahead], st);
            st = st1;
            slot = slot1;
            buf ^= 1;
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        // empty sequences leave with what entered them
        if (g.leave)
            for (int64_t s = blockIdx.x; s < g.q.n_seq; s += gridDim.x)
                if (g.q.at(s + 1) <= g.q.at(s))
                    for (int64_t c = r.tid; c < g.n_chan; c += P::NC)
                        g.leave[s * g.n_chan + c] = g.enter ? g.enter[s * g.n_chan + c] : A(0);
    } else if (r.tid < P::NC + P::NSCAN) {                 // scan warps
        int slot = 0, buf = 0;
        for (;;) {
            bar_sync(BAR_P1 + buf, P::NC + P::NSCAN);
            if (sm.plan[slot].tile < 0)
                break;
            r.scan(sm.plan[slot], slot, buf, r.warp - P::NW);
            __syncwarp();
            bar_arrive(BAR_P2 + buf, P::NC + P::NSCAN);
            slot = slot + 1 == NP ? 0 : slot + 1;
            buf ^= 1;
        }
    } else {                                               // plan warp
        // the compute warps take NS plans before their loop and one in every turn of it
        int slot = 0, end = INT32_MAX;
        for (int j = 0; j < end; ++j) {
            if (end == INT32_MAX) {
                if (!r.plan(slot, j))
                    end = j + NS;
            } else if (r.lane == 0)
                sm.plan[slot].tile = -1;
            __syncwarp();
            bar_sync(BAR_PLAN, P::NC + 32);
            slot = slot + 1 == NP ? 0 : slot + 1;
        }
    }
}

// ------------------------------------------------------------------ launch
int sm_count();

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

// The widest unit of channels that every array's rows are aligned to: 16 bytes, 4 bytes (two of a 16-bit
// type) or one value.  Copies below 4 bytes are not asynchronous.
template <typename S, int GATE, bool REV>
sla_status launch_recur(RecurArgs<S> &g, cudaStream_t s)
{
    uintptr_t bits = 0;
    for (int k = 0; k < 4; ++k)
        if (g.in[k])
            bits |= (uintptr_t)g.in[k] | (uintptr_t)(g.ldin[k] * (int64_t)sizeof(S));
    for (int k = 0; k < 2; ++k)
        if (g.out[k])
            bits |= (uintptr_t)g.out[k] | (uintptr_t)(g.ldout[k] * (int64_t)sizeof(S));
    if (bits % 16 == 0)
        return launch_recur_u<S, GATE, 16 / (int)sizeof(S), REV>(g, s);
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
