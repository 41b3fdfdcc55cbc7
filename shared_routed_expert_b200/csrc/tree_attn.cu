// Attention of new tokens (decode rows, drafted chains and trees, prefill chunks)
// over a paged cache:
//   s_j = softmax_scale * q . k_j over the keys a row sees, m = max s, p_j = e^{s_j - m},
//   out = sum p_j v_j / sum p_j,  lse = m + ln sum p_j.
#include "kernels.cuh"
#include "tree_attn.cuh"

namespace sre {

namespace {

constexpr int RW_WARPS = 4;

// One warp per (row, query head), key by key.
template <int EPL, bool F8>
__global__ void __launch_bounds__(RW_WARPS * 32) rows_kernel(const AttnArgs a) {
    const int lane = threadIdx.x & 31;
    const int b = blockIdx.y;
    const SeqInfo s = seq_info(a.c, b, a.T, attn_max_new(a));
    if (!s.ok) {
        if (blockIdx.x == 0 && threadIdx.x == 0) report(a.status, MOE_ERR_DEVICE, b);
        return;
    }
    for (long long it = static_cast<long long>(blockIdx.x) * RW_WARPS + (threadIdx.x >> 5);
         it < static_cast<long long>(s.n) * a.n_q; it += static_cast<long long>(gridDim.x) * RW_WARPS) {
        const int i = static_cast<int>(it / a.n_q), h = static_cast<int>(it % a.n_q);
        const long long t = s.row0 + i;
        float q[EPL], acc[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            q[j] = bf16_to_f32(a.q[t * a.q_stride + h * (32 * EPL) + lane * EPL + j]);
            acc[j] = 0.f;
        }
        float m = -INFINITY, l = 0.f;
        const int hi = s.ctx + (a.mask != nullptr ? s.n : i + 1);
        attend_row<EPL, F8>(a, b, s, i, h / a.group, q, 0, hi, m, l, acc, lane);
        const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            a.out[t * a.out_stride + h * (32 * EPL) + lane * EPL + j] =
                f32_to_bf16(l == 0.f ? 0.f : acc[j] * inv * a.c.v_scale);
        if (a.lse != nullptr && lane == 0)
            a.lse[t * a.n_q + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2F;
    }
}

template <int EPL>
void rows_epl(const AttnArgs& a, dim3 grid, cudaStream_t st) {
    if (a.f8) rows_kernel<EPL, true><<<grid, RW_WARPS * 32, 0, st>>>(a);
    else rows_kernel<EPL, false><<<grid, RW_WARPS * 32, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_tree_attn_rows(const AttnArgs& a, cudaStream_t st) {
    ProfileScope ps("tree_attention", st);
    const long long items = (static_cast<long long>(a.c.max_new) * a.n_q + RW_WARPS - 1) / RW_WARPS;
    const dim3 grid(static_cast<unsigned>(items < 65536 ? items : 65536), a.c.B);
    if (a.head_dim == 64) rows_epl<2>(a, grid, st);
    else if (a.head_dim == 128) rows_epl<4>(a, grid, st);
    else rows_epl<8>(a, grid, st);
    note_launch();
    return cudaGetLastError();
}

}  // namespace sre
