// Gated linear recurrence h_t = a_t h_{t-1} + w_t b_t over packed sequences: the solve with a unit
// lower bidiagonal matrix, its adjoint (the solve with the transpose, and the gradient on the
// subdiagonal), and the single-row step on a pool of states.
#include <cuda_runtime.h>

#include <algorithm>

#include "seq_rows.cuh"

namespace sla {
namespace {

constexpr int RT = 128;

struct SeqBounds {
    const int32_t *off;   // NULL: equal lengths
    int64_t n_tokens;
    int32_t n_seq;
    // Offsets are read from the device and clamped, so that no offset leads outside the rows.
    __device__ __forceinline__ int64_t at(int64_t s) const
    {
        if (!off)
            return n_tokens / n_seq * s;
        const int64_t v = off[s];
        return v < 0 ? 0 : v > n_tokens ? n_tokens : v;
    }
};

template <typename S, int GATE>
__global__ void __launch_bounds__(RT) k_recur_solve(SeqBounds q, int64_t n_chan, const S *a, int64_t lda, const S *b,
                                                    int64_t ldb, const typename RowType<S>::A *h0, S *h, int64_t ldh,
                                                    typename RowType<S>::A *last)
{
    using R = RowType<S>;
    using A = typename R::A;
    const int64_t c = (int64_t)blockIdx.x * RT + threadIdx.x;
    if (c >= n_chan)
        return;
    for (int64_t s = blockIdx.y; s < q.n_seq; s += gridDim.y) {
        const int64_t t0 = q.at(s), t1 = q.at(s + 1);
        A v = h0 ? h0[s * n_chan + c] : A(0);
        for (int64_t t = t0; t < t1; ++t) {
            A ca, w;
            gate_of<GATE>(R::up(a[t * lda + c]), ca, w);
            const A u = w * R::up(b[t * ldb + c]);
            v = (t == t0 && !h0) ? u : fma_of(ca, v, u);
            h[t * ldh + c] = R::down(v);
        }
        if (last)
            last[s * n_chan + c] = v;
    }
}

template <typename S, int GATE>
__global__ void __launch_bounds__(RT)
    k_recur_adjoint(SeqBounds q, int64_t n_chan, const S *a, int64_t lda, const S *b, int64_t ldb, const S *h,
                    int64_t ldh, const typename RowType<S>::A *h0, const S *dh, int64_t lddh,
                    const typename RowType<S>::A *dlast, S *dz, int64_t lddz, S *db, int64_t lddb,
                    typename RowType<S>::A *dh0)
{
    using R = RowType<S>;
    using A = typename R::A;
    const int64_t c = (int64_t)blockIdx.x * RT + threadIdx.x;
    if (c >= n_chan)
        return;
    for (int64_t s = blockIdx.y; s < q.n_seq; s += gridDim.y) {
        const int64_t t0 = q.at(s), t1 = q.at(s + 1);
        // lambda_t = g_t + a_{t+1} lambda_{t+1} by one fused multiply-add, written out so that every
        // variant of the loop rounds alike
        A next = A(1), lam = dlast ? dlast[s * n_chan + c] : A(0);
        for (int64_t t = t1 - 1; t >= t0; --t) {
            A ca, w;
            gate_of<GATE>(R::up(a[t * lda + c]), ca, w);
            lam = fma_of(next, lam, dh ? R::up(dh[t * lddh + c]) : A(0));
            const bool first = t == t0;
            const A before = !first ? R::up(h[(t - 1) * ldh + c]) : h0 ? h0[s * n_chan + c] : A(0);
            if (db)
                db[t * lddb + c] = R::down(w * lam);
            if (dz) {
                A d;
                if constexpr (GATE == SLA_GATE_VALUE)
                    d = lam * before;
                else if constexpr (GATE == SLA_GATE_EXP)
                    d = lam * before * ca;
                else {
                    const A u = R::up(b[t * ldb + c]);
                    // without a first state the first row is w b alone: its coefficient still weighs b
                    d = lam * (before - u) * ca * w;
                }
                dz[t * lddz + c] = R::down(d);
            }
            next = ca;
        }
        if (dh0)
            dh0[s * n_chan + c] = next * lam;
    }
}

// Zeros in the rows in front of the first sequence and behind the last one.
template <typename S>
__global__ void __launch_bounds__(RT) k_recur_fill(SeqBounds q, int64_t n_chan, S *x, int64_t ldx)
{
    const int64_t c = (int64_t)blockIdx.x * RT + threadIdx.x;
    if (c >= n_chan)
        return;
    const int64_t lo = q.at(0), hi = max(lo, q.at(q.n_seq));
    for (int64_t t = blockIdx.y; t < q.n_tokens; t += gridDim.y)
        if (t < lo || t >= hi)
            x[t * ldx + c] = S(0.0f);
}

template <typename S, int GATE>
__global__ void __launch_bounds__(RT)
    k_recur_step(int64_t n_rows, int64_t n_chan, int64_t n_slots, const S *a, int64_t lda, const S *b, int64_t ldb,
                 typename RowType<S>::A *state, int64_t lds, const int32_t *index, S *h, int64_t ldh, int fill)
{
    using R = RowType<S>;
    using A = typename R::A;
    const int64_t c = (int64_t)blockIdx.x * RT + threadIdx.x;
    if (c >= n_chan)
        return;
    for (int64_t r = blockIdx.y; r < n_rows; r += gridDim.y) {
        const int64_t i = index ? index[r] : r;
        if (i < 0 || i >= n_slots) {
            if (fill)
                h[r * ldh + c] = S(0.0f);
            continue;
        }
        A ca, w;
        gate_of<GATE>(R::up(a[r * lda + c]), ca, w);
        const A v = fma_of(ca, state[i * lds + c], w * R::up(b[r * ldb + c]));
        state[i * lds + c] = v;
        h[r * ldh + c] = R::down(v);
    }
}

sla_status check_common(int32_t dtype, int32_t gate, int64_t n_rows, int64_t n_chan, uint32_t flags)
{
    if (!row_dtype_ok(dtype))
        return fail(SLA_ERR_INVALID_ARG, "dtype must be SLA_F32, SLA_F64, SLA_BF16 or SLA_F16");
    if (gate < SLA_GATE_VALUE || gate > SLA_GATE_SIGMOID)
        return fail(SLA_ERR_INVALID_ARG, "unknown gate");
    if (n_rows < 0 || n_rows > INT32_MAX || n_chan < 0 || n_chan > INT32_MAX)
        return fail(SLA_ERR_INVALID_ARG, "rows and channels must be within [0, 2^31)");
    if (flags & ~SLA_FILL_REST)
        return fail(SLA_ERR_INVALID_ARG, "unknown flags");
    return SLA_SUCCESS;
}

sla_status check_in(const void *p, int64_t ld, int64_t n_chan)
{
    if (!p || (ld != 0 && ld < n_chan))
        return fail(SLA_ERR_INVALID_ARG, "NULL input rows, or a row stride below the number of channels");
    return SLA_SUCCESS;
}

sla_status check_out(const void *p, int64_t ld, int64_t n_chan)
{
    if (!p || ld < n_chan)
        return fail(SLA_ERR_INVALID_ARG, "NULL output rows, or a row stride below the number of channels");
    return SLA_SUCCESS;
}

sla_status check_seqs(int64_t n_tokens, int32_t n_seq, const int32_t *d_seq_off)
{
    if (n_seq < 0)
        return fail(SLA_ERR_INVALID_ARG, "n_seq must not be negative");
    if (!d_seq_off && (n_seq == 0 ? n_tokens != 0 : n_tokens % n_seq != 0))
        return fail(SLA_ERR_INVALID_ARG, "without offsets n_tokens must be a multiple of n_seq");
    return SLA_SUCCESS;
}

template <class F>
sla_status with_gate(int32_t gate, F f)
{
    switch (gate) {
    case SLA_GATE_VALUE: return f(std::integral_constant<int, SLA_GATE_VALUE>());
    case SLA_GATE_EXP: return f(std::integral_constant<int, SLA_GATE_EXP>());
    default: return f(std::integral_constant<int, SLA_GATE_SIGMOID>());
    }
}

dim3 grid_of(int64_t n_chan, int64_t rows)
{
    return dim3((unsigned)((n_chan + RT - 1) / RT), (unsigned)std::max<int64_t>(1, std::min<int64_t>(rows, 32768)));
}

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

size_t sla_recur_workspace_bytes(int32_t dtype, int64_t n_tokens, int64_t n_chan)
{
    (void)dtype;
    (void)n_tokens;
    (void)n_chan;
    return 0;
}

sla_status sla_recur_solve(int32_t dtype, int32_t gate, int64_t n_tokens, int64_t n_chan, int32_t n_seq,
                           const int32_t *d_seq_off, const void *d_a, int64_t lda, const void *d_b, int64_t ldb,
                           const void *d_h0, void *d_h, int64_t ldh, void *d_h_last, uint32_t flags, void *d_work,
                           size_t work_bytes, void *stream)
{
    SLA_TRY(check_common(dtype, gate, n_tokens, n_chan, flags));
    SLA_TRY(check_seqs(n_tokens, n_seq, d_seq_off));
    if (n_chan == 0 || (n_tokens == 0 && n_seq == 0))
        return SLA_SUCCESS;
    if (n_tokens > 0) {
        SLA_TRY(check_in(d_a, lda, n_chan));
        SLA_TRY(check_in(d_b, ldb, n_chan));
        SLA_TRY(check_out(d_h, ldh, n_chan));
    }
    if (work_bytes < sla_recur_workspace_bytes(dtype, n_tokens, n_chan))
        return fail(SLA_ERR_INVALID_ARG, "d_work is too small");
    cudaStream_t s = (cudaStream_t)stream;
    const SeqBounds q{d_seq_off, n_tokens, n_seq};
    return with_row_type(dtype, [&](auto tag) {
        using S = decltype(tag);
        using A = typename RowType<S>::A;
        if (flags & SLA_FILL_REST)
            k_recur_fill<S><<<grid_of(n_chan, n_tokens), RT, 0, s>>>(q, n_chan, (S *)d_h, ldh);
        return with_gate(gate, [&](auto g) {
            k_recur_solve<S, decltype(g)::value><<<grid_of(n_chan, n_seq), RT, 0, s>>>(
                q, n_chan, (const S *)d_a, lda, (const S *)d_b, ldb, (const A *)d_h0, (S *)d_h, ldh, (A *)d_h_last);
            SLA_CUDA_TRY(cudaGetLastError());
            return (sla_status)SLA_SUCCESS;
        });
    });
}

sla_status sla_recur_adjoint(int32_t dtype, int32_t gate, int64_t n_tokens, int64_t n_chan, int32_t n_seq,
                             const int32_t *d_seq_off, const void *d_a, int64_t lda, const void *d_b, int64_t ldb,
                             const void *d_h, int64_t ldh, const void *d_h0, const void *d_dh, int64_t lddh,
                             const void *d_dh_last, void *d_dz, int64_t lddz, void *d_db, int64_t lddb, void *d_dh0,
                             uint32_t flags, void *d_work, size_t work_bytes, void *stream)
{
    SLA_TRY(check_common(dtype, gate, n_tokens, n_chan, flags));
    SLA_TRY(check_seqs(n_tokens, n_seq, d_seq_off));
    if (d_dh0 && !d_h0)
        return fail(SLA_ERR_INVALID_ARG, "d_dh0 needs d_h0");
    if (n_chan == 0 || (n_tokens == 0 && n_seq == 0))
        return SLA_SUCCESS;
    if (n_tokens > 0) {
        SLA_TRY(check_in(d_a, lda, n_chan));
        if (gate == SLA_GATE_SIGMOID && d_dz)
            SLA_TRY(check_in(d_b, ldb, n_chan));
        if (d_dz)
            SLA_TRY(check_in(d_h, ldh, n_chan));
        if (d_dh)
            SLA_TRY(check_in(d_dh, lddh, n_chan));
        if (d_dz)
            SLA_TRY(check_out(d_dz, lddz, n_chan));
        if (d_db)
            SLA_TRY(check_out(d_db, lddb, n_chan));
    }
    if (work_bytes < sla_recur_workspace_bytes(dtype, n_tokens, n_chan))
        return fail(SLA_ERR_INVALID_ARG, "d_work is too small");
    cudaStream_t s = (cudaStream_t)stream;
    const SeqBounds q{d_seq_off, n_tokens, n_seq};
    return with_row_type(dtype, [&](auto tag) {
        using S = decltype(tag);
        using A = typename RowType<S>::A;
        if (flags & SLA_FILL_REST) {
            if (d_dz)
                k_recur_fill<S><<<grid_of(n_chan, n_tokens), RT, 0, s>>>(q, n_chan, (S *)d_dz, lddz);
            if (d_db)
                k_recur_fill<S><<<grid_of(n_chan, n_tokens), RT, 0, s>>>(q, n_chan, (S *)d_db, lddb);
        }
        return with_gate(gate, [&](auto g) {
            k_recur_adjoint<S, decltype(g)::value><<<grid_of(n_chan, n_seq), RT, 0, s>>>(
                q, n_chan, (const S *)d_a, lda, (const S *)d_b, ldb, (const S *)d_h, ldh, (const A *)d_h0,
                (const S *)d_dh, lddh, (const A *)d_dh_last, (S *)d_dz, lddz, (S *)d_db, lddb, (A *)d_dh0);
            SLA_CUDA_TRY(cudaGetLastError());
            return (sla_status)SLA_SUCCESS;
        });
    });
}

sla_status sla_recur_step(int32_t dtype, int32_t gate, int64_t n_rows, int64_t n_chan, int64_t n_slots,
                          const void *d_a, int64_t lda, const void *d_b, int64_t ldb, void *d_state, int64_t ldstate,
                          const int32_t *d_index, void *d_h, int64_t ldh, uint32_t flags, void *stream)
{
    SLA_TRY(check_common(dtype, gate, n_rows, n_chan, flags));
    if (n_slots < 0 || n_slots > INT32_MAX)
        return fail(SLA_ERR_INVALID_ARG, "slots must be within [0, 2^31)");
    if (n_rows == 0 || n_chan == 0)
        return SLA_SUCCESS;
    SLA_TRY(check_in(d_a, lda, n_chan));
    SLA_TRY(check_in(d_b, ldb, n_chan));
    SLA_TRY(check_out(d_h, ldh, n_chan));
    if (n_slots > 0)
        SLA_TRY(check_out(d_state, ldstate, n_chan));
    cudaStream_t s = (cudaStream_t)stream;
    return with_row_type(dtype, [&](auto tag) {
        using S = decltype(tag);
        using A = typename RowType<S>::A;
        return with_gate(gate, [&](auto g) {
            k_recur_step<S, decltype(g)::value><<<grid_of(n_chan, n_rows), RT, 0, s>>>(
                n_rows, n_chan, n_slots, (const S *)d_a, lda, (const S *)d_b, ldb, (A *)d_state, ldstate, d_index,
                (S *)d_h, ldh, (flags & SLA_FILL_REST) != 0);
            SLA_CUDA_TRY(cudaGetLastError());
            return (sla_status)SLA_SUCCESS;
        });
    });
}

}  // extern "C"
