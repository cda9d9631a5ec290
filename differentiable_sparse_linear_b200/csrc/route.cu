// Routing of tokens to experts: the plan (a stable counting sort of the entries by expert) and the
// products with the routing matrix R (tokens x slots, one entry per used slot), its transpose and the
// gradient on its pattern.
#include <cuda_runtime.h>

#include <algorithm>

#include "seq_rows.cuh"

namespace sla {
namespace {

constexpr int MAX_EXPERTS = 4096;
constexpr int RT = 128;

// ------------------------------------------------------------------ sort
template <typename I>
__device__ __forceinline__ int expert_of(const I *ids, int64_t e, int n_experts)
{
    const I v = ids[e];
    return v >= 0 && v < (I)n_experts ? (int)v : -1;
}

// One block.  Warp w owns a contiguous run of entries; cnt[w][x] is first its number of entries of
// expert x, then the slot its next entry of x gets.  Equal experts among a warp's 32 entries are
// ranked by lane, so the order within an expert is the order of the entries' numbers.
template <typename I>
__global__ void __launch_bounds__(1024)
    k_route_sort_one(int64_t n, int n_experts, int align, const I *ids, int64_t n_slots, int32_t *offsets,
                     int32_t *counts, int32_t *entry, int32_t *slot)
{
    extern __shared__ int cnt[];
    __shared__ int s_total;
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < warps * n_experts; i += blockDim.x)
        cnt[i] = 0;
    for (int64_t i = threadIdx.x; i < n_slots; i += blockDim.x)
        entry[i] = -1;
    __syncthreads();
    const int64_t per = ((n + warps - 1) / warps + 31) / 32 * 32;
    const int64_t e0 = min(n, per * warp), e1 = min(n, e0 + per);
    for (int64_t e = e0 + lane; e < e1; e += 32) {
        const int x = expert_of(ids, e, n_experts);
        if (x >= 0)
            atomicAdd(&cnt[warp * n_experts + x], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        int at = 0;
        for (int x = 0; x < n_experts; ++x) {
            offsets[x] = at;
            int next = at;
            for (int w = 0; w < warps; ++w) {
                const int c = cnt[w * n_experts + x];
                cnt[w * n_experts + x] = next;
                next += c;
            }
            counts[x] = next - at;
            at += (next - at + align - 1) / align * align;
        }
        offsets[n_experts] = at;
        s_total = at;
    }
    __syncthreads();
    for (int64_t e = e0; e < e1; e += 32) {
        const int x = e + lane < e1 ? expert_of(ids, e + lane, n_experts) : -2;
        const unsigned peers = __match_any_sync(0xffffffffu, x);
        if (x >= 0) {
            const int rank = __popc(peers & ((1u << lane) - 1));
            const int p = cnt[warp * n_experts + x] + rank;
            slot[e + lane] = p;
            entry[p] = (int)(e + lane);
        } else if (x == -1)
            slot[e + lane] = -1;
        __syncwarp();
        if (x >= 0 && (peers >> lane) == 1)   // the last of its kind in the warp
            cnt[warp * n_experts + x] += __popc(peers);
        __syncwarp();
    }
}

// ------------------------------------------------------------------ products
// Rows of the slot side that belong to no entry: padding of the experts (zeros), and with `fill`
// the slots behind the last expert's.
template <typename S>
__global__ void __launch_bounds__(RT) k_route_padding(int n_experts, int64_t n_slots, int64_t n_chan,
                                                      const int32_t *offsets, const int32_t *counts, S *xs,
                                                      int64_t ldxs, int fill)
{
    // experts, then the rest
    for (int x = blockIdx.x; x <= n_experts; x += gridDim.x) {
        int64_t r0, r1;
        if (x < n_experts) {
            r0 = (int64_t)offsets[x] + counts[x];
            r1 = offsets[x + 1];
        } else {
            r0 = offsets[n_experts];
            r1 = fill ? n_slots : r0;
        }
        r0 = max(r0, (int64_t)0);
        r1 = min(r1, n_slots);
        for (int64_t r = r0; r < r1; ++r)
            for (int64_t c = threadIdx.x; c < n_chan; c += RT)
                xs[r * ldxs + c] = S(0.0f);
    }
}

// R^T x: one block per token writes its row to each of its slots.
template <typename S>
__global__ void __launch_bounds__(RT)
    k_route_to_slots(int64_t n_tokens, int top_k, int64_t n_slots, int64_t n_chan, const S *x, int64_t ldx,
                     const int32_t *slot, const typename RowType<S>::A *weight, S *xs, int64_t ldxs)
{
    using R = RowType<S>;
    for (int64_t t = blockIdx.x; t < n_tokens; t += gridDim.x)
        for (int j = 0; j < top_k; ++j) {
            const int64_t p = slot[t * top_k + j];
            if (p < 0 || p >= n_slots)
                continue;
            for (int64_t c = threadIdx.x; c < n_chan; c += RT) {
                const S v = x[t * ldx + c];
                xs[p * ldxs + c] = weight ? R::down(weight[t * top_k + j] * R::up(v)) : v;
            }
        }
}

// R xs: one block per token sums its slots' rows.
template <typename S>
__global__ void __launch_bounds__(RT)
    k_route_to_tokens(int64_t n_tokens, int top_k, int64_t n_slots, int64_t n_chan, const S *xs, int64_t ldxs,
                      const int32_t *slot, const typename RowType<S>::A *weight, S *y, int64_t ldy)
{
    using R = RowType<S>;
    using A = typename R::A;
    for (int64_t t = blockIdx.x; t < n_tokens; t += gridDim.x)
        for (int64_t c = threadIdx.x; c < n_chan; c += RT) {
            A v = A(0);
            for (int j = 0; j < top_k; ++j) {
                const int64_t p = slot[t * top_k + j];
                if (p < 0 || p >= n_slots)
                    continue;
                const A u = R::up(xs[p * ldxs + c]);
                v = weight ? fma_of(weight[t * top_k + j], u, v) : v + u;
            }
            y[t * ldy + c] = R::down(v);
        }
}

// The gradient on the pattern: one warp per entry.
template <typename S>
__global__ void __launch_bounds__(RT)
    k_route_pattern(int64_t n_tokens, int top_k, int64_t n_slots, int64_t n_chan, const S *x, int64_t ldx, const S *xs,
                    int64_t ldxs, const int32_t *slot, typename RowType<S>::A *dweight)
{
    using R = RowType<S>;
    using A = typename R::A;
    const int lane = threadIdx.x & 31;
    const int64_t n = n_tokens * top_k;
    for (int64_t e = (int64_t)blockIdx.x * (RT / 32) + (threadIdx.x >> 5); e < n; e += (int64_t)gridDim.x * (RT / 32)) {
        const int64_t p = slot[e], t = e / top_k;
        A v = A(0);
        if (p >= 0 && p < n_slots)
            for (int64_t c = lane; c < n_chan; c += 32)
                v = fma_of(R::up(x[t * ldx + c]), R::up(xs[p * ldxs + c]), v);
        for (int o = 16; o > 0; o >>= 1)
            v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0)
            dweight[e] = v;
    }
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
    if (n_rows == 0)
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

unsigned blocks_for(int64_t n) { return (unsigned)std::max<int64_t>(1, std::min<int64_t>(n, 1 << 20)); }

}  // namespace
}  // namespace sla

using namespace sla;

extern "C" {

size_t sla_route_workspace_bytes(int64_t n_tokens, int32_t top_k, int32_t n_experts)
{
    (void)n_tokens;
    (void)top_k;
    (void)n_experts;
    return 0;
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
    if (work_bytes < sla_route_workspace_bytes(n_tokens, top_k, n_experts))
        return fail(SLA_ERR_INVALID_ARG, "d_work is too small");
    cudaStream_t s = (cudaStream_t)stream;
    const int warps = std::max(1, std::min(32, (128 << 10) / (4 * n_experts)));
    const size_t smem = sizeof(int) * (size_t)warps * n_experts;
    auto launch = [&](auto kernel, auto ids) -> sla_status {
        SLA_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 128 << 10));
        kernel<<<1, 32 * warps, smem, s>>>(n, n_experts, align, ids, n_slots, d_offsets, d_counts, d_entry, d_slot);
        SLA_CUDA_TRY(cudaGetLastError());
        return SLA_SUCCESS;
    };
    return id_bytes == 4 ? launch(k_route_sort_one<int32_t>, (const int32_t *)d_expert)
                         : launch(k_route_sort_one<int64_t>, (const int64_t *)d_expert);
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
    cudaStream_t s = (cudaStream_t)stream;
    return with_row_type(dtype, [&](auto tag) {
        using S = decltype(tag);
        using A = typename RowType<S>::A;
        k_route_to_tokens<S><<<blocks_for(n_tokens), RT, 0, s>>>(n_tokens, top_k, n_slots, n_chan, (const S *)d_dxs,
                                                                 lddxs, d_slot, (const A *)d_weight, (S *)d_dx, lddx);
        if (d_dweight)
            k_route_pattern<S><<<blocks_for(n_tokens), RT, 0, s>>>(n_tokens, top_k, n_slots, n_chan, (const S *)d_x,
                                                                   ldx, (const S *)d_dxs, lddxs, d_slot,
                                                                   (A *)d_dweight);
        SLA_CUDA_TRY(cudaGetLastError());
        return (sla_status)SLA_SUCCESS;
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
    cudaStream_t s = (cudaStream_t)stream;
    return with_row_type(dtype, [&](auto tag) {
        using S = decltype(tag);
        using A = typename RowType<S>::A;
        k_route_padding<S><<<blocks_for(n_experts + 1), RT, 0, s>>>(n_experts, n_slots, n_chan, d_offsets, d_counts,
                                                                    (S *)d_dys, lddys, (flags & SLA_FILL_REST) != 0);
        if (n_tokens > 0)
            k_route_to_slots<S><<<blocks_for(n_tokens), RT, 0, s>>>(n_tokens, top_k, n_slots, n_chan, (const S *)d_dy,
                                                                    lddy, d_slot, (const A *)d_weight, (S *)d_dys,
                                                                    lddys);
        if (d_dweight && n_tokens > 0)
            k_route_pattern<S><<<blocks_for(n_tokens), RT, 0, s>>>(n_tokens, top_k, n_slots, n_chan, (const S *)d_dy,
                                                                   lddy, (const S *)d_ys, ldys, d_slot,
                                                                   (A *)d_dweight);
        SLA_CUDA_TRY(cudaGetLastError());
        return (sla_status)SLA_SUCCESS;
    });
}

}  // extern "C"
