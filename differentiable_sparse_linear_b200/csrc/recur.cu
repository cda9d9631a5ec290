// Gated linear recurrence h_t = a_t h_{t-1} + w_t b_t over packed sequences: the entry points of the solve
// with a unit lower bidiagonal matrix and of its adjoint (recur_core.cuh), and the single-row step
// on a pool of states.
#include "recur_core.cuh"

namespace sla {
namespace {

constexpr int RT = 128;

// One row for each sequence of a serving batch.  A thread takes V channels of a row: 16 bytes of a, b and h where
// everything is aligned to it, one value otherwise.  Bound by memory: 3 values and a state in and out a channel;
// 384 x 4096 bf16 take 4.3 us (22 MB, floor 3.4), one value a thread took 8.8.
template <typename S, int GATE, int V>
__global__ void __launch_bounds__(RT)
    k_recur_step(int64_t n_rows, int64_t n_chan, int64_t n_slots, const S *a, int64_t lda, const S *b, int64_t ldb,
                 typename RowType<S>::A *state, int64_t lds, const int32_t *index, S *h, int64_t ldh, int fill)
{
    using R = RowType<S>;
    using A = typename R::A;
    const int64_t c = ((int64_t)blockIdx.x * RT + threadIdx.x) * V;
    if (c >= n_chan)
        return;
    for (int64_t r = blockIdx.y; r < n_rows; r += gridDim.y) {
        const int64_t i = index ? index[r] : r;
        const bool live = i >= 0 && i < n_slots;
        if (!live && !fill)
            continue;
        constexpr int N = V > 1 ? V : 2;                   // arithmetic goes in pairs
        A x[N] = {};
        if (live) {
            A z[N] = {}, u[N] = {}, w[N], v[N] = {};
            A *st = state + i * lds + c;
            if constexpr (V > 1) {
                const uint4 ra = *reinterpret_cast<const uint4 *>(a + r * lda + c), rb = *reinterpret_cast<const uint4 *>(b + r * ldb + c);
                uint4 rs[V * sizeof(A) / 16];
#pragma unroll
                for (int k = 0; k < (int)(V * sizeof(A) / 16); ++k)
                    rs[k] = reinterpret_cast<const uint4 *>(st)[k];
                unpack16(ra, z, S());
                unpack16(rb, u, S());
                memcpy(v, rs, sizeof(rs));
            } else {
                z[0] = R::up(a[r * lda + c]);
                u[0] = R::up(b[r * ldb + c]);
                v[0] = st[0];
            }
            gates_of<GATE, sizeof(S) == 2>(z, z, w);
            vmul(u, w, u);
            vfma(x, z, v, u);
            if constexpr (V > 1) {
                uint4 rs[V * sizeof(A) / 16];
                memcpy(rs, x, sizeof(rs));
#pragma unroll
                for (int k = 0; k < (int)(V * sizeof(A) / 16); ++k)
                    reinterpret_cast<uint4 *>(st)[k] = rs[k];
            } else
                st[0] = x[0];
        }
        if constexpr (V > 1)
            *reinterpret_cast<uint4 *>(h + r * ldh + c) = pack16(x, S());
        else
            h[r * ldh + c] = R::down(x[0]);
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

sla_status check_work(int32_t dtype, int64_t n_tokens, int64_t n_chan, const void *d_work, size_t work_bytes)
{
    const size_t need = sla_recur_workspace_bytes(dtype, n_tokens, n_chan);
    if (need && (!d_work || work_bytes < need || (uintptr_t)d_work % 16))
        return fail(SLA_ERR_INVALID_ARG, "d_work is NULL, smaller than sla_recur_workspace_bytes or not 16-byte aligned");
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

dim3 grid_of(int64_t n_chan, int64_t rows)
{
    return dim3((unsigned)((n_chan + RT - 1) / RT), (unsigned)std::max<int64_t>(1, std::min<int64_t>(rows, 32768)));
}

}  // namespace

EncodeTiled encode_tiled()
{
    static const EncodeTiled found = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult got;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &got);
        if (e != cudaSuccess || got != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            p = nullptr;
        }
        return (EncodeTiled)p;
    }();
    return found;
}

int sm_count()
{
    static std::atomic<int> known[64];                     // per device; 0: not asked yet
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return 148;
    if (dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0)
        return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
        return 148;
    if (dev < 64)
        known[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace sla

using namespace sla;

extern "C" {

size_t sla_recur_workspace_bytes(int32_t dtype, int64_t n_tokens, int64_t n_chan)
{
    if (!row_dtype_ok(dtype) || n_tokens <= 0 || n_chan <= 0 || n_tokens > INT32_MAX || n_chan > INT32_MAX)
        return 0;
    // the tiles of the adjoint with the sigmoid gate are the shortest ones
    return dtype == SLA_F64 ? RecurWork<double, SLA_GATE_SIGMOID, true>::bytes(n_tokens, n_chan)
                            : RecurWork<float, SLA_GATE_SIGMOID, true>::bytes(n_tokens, n_chan);
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
    SLA_TRY(check_work(dtype, n_tokens, n_chan, d_work, work_bytes));
    return with_row_type(dtype, [&](auto tag) {
        using S = decltype(tag);
        using A = typename RowType<S>::A;
        RecurArgs<S> g{};
        g.q = SeqBounds{d_seq_off, n_tokens, n_seq};
        g.n_chan = n_chan;
        g.in[0] = (const S *)d_a;
        g.in[1] = (const S *)d_b;
        g.ldin[0] = lda;
        g.ldin[1] = ldb;
        g.out[0] = (S *)d_h;
        g.ldout[0] = ldh;
        g.enter = (const A *)d_h0;
        g.leave = (A *)d_h_last;
        g.fill = (flags & SLA_FILL_REST) != 0;
        return recur_forward(dtype, gate, &g, d_work, (cudaStream_t)stream);
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
    SLA_TRY(check_work(dtype, n_tokens, n_chan, d_work, work_bytes));
    return with_row_type(dtype, [&](auto tag) {
        using S = decltype(tag);
        using A = typename RowType<S>::A;
        RecurArgs<S> g{};
        g.q = SeqBounds{d_seq_off, n_tokens, n_seq};
        g.n_chan = n_chan;
        g.in[0] = (const S *)d_a;
        g.ldin[0] = lda;
        g.in[1] = (const S *)d_dh;
        g.ldin[1] = lddh;
        if (d_dz) {
            g.in[2] = (const S *)d_h;
            g.ldin[2] = ldh;
            if (gate == SLA_GATE_SIGMOID) {
                g.in[3] = (const S *)d_b;
                g.ldin[3] = ldb;
            }
        }
        g.out[0] = (S *)d_db;
        g.ldout[0] = lddb;
        g.out[1] = (S *)d_dz;
        g.ldout[1] = lddz;
        g.enter = (const A *)d_dh_last;
        g.before = (const A *)d_h0;
        g.leave = (A *)d_dh0;
        g.fill = (flags & SLA_FILL_REST) != 0;
        return recur_backward(dtype, gate, &g, d_work, (cudaStream_t)stream);
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
            constexpr int GATE = decltype(g)::value, V = 16 / (int)sizeof(S);
            const uintptr_t bits = (uintptr_t)d_a | (uintptr_t)d_b | (uintptr_t)d_h | (uintptr_t)d_state |
                                   (uintptr_t)((lda | ldb | ldh | n_chan) * (int64_t)sizeof(S)) |
                                   (uintptr_t)(ldstate * (int64_t)sizeof(A));
            auto run = [&](auto kernel, int v) {
                kernel<<<grid_of((n_chan + v - 1) / v, n_rows), RT, 0, s>>>(
                    n_rows, n_chan, n_slots, (const S *)d_a, lda, (const S *)d_b, ldb, (A *)d_state, ldstate, d_index,
                    (S *)d_h, ldh, (flags & SLA_FILL_REST) != 0);
            };
            if (bits % 16 == 0)
                run(k_recur_step<S, GATE, V>, V);
            else
                run(k_recur_step<S, GATE, 1>, 1);
            SLA_CUDA_TRY(cudaGetLastError());
            return (sla_status)SLA_SUCCESS;
        });
    });
}

}  // extern "C"
