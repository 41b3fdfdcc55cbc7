// Attention of new tokens (decode rows, drafted chains and trees, prefill chunks)
// over a paged cache:
//   s_j = softmax_scale * q . k_j over the keys a row sees, m = max s, p_j = e^{s_j - m},
//   out = sum p_j v_j / sum p_j,  lse = m + ln sum p_j.
// Here: the join of partial results, and the cache's TMA maps.
#include "kernels.cuh"
#include "tree_attn.cuh"

namespace sre {

namespace {

constexpr int JN_WARPS = 4;

// Joins the items that a cut between two shares goes through: block x looks at the cut
// in front of share x + 1 and, if that cut is the first inside its item, joins the
// item's parts: with M = max m_p, sum_p 2^{m_p - M} (l_p, o_p), in the order of the keys.
// Bound by latency (a few hundred KB out of L2).
template <int EPL>
__global__ void __launch_bounds__(JN_WARPS * 32) join_kernel(const AttnArgs a, const Tiling g, const Partials p, int blocks,
                                                             int least) {
    __shared__ ScanShared scan;
    long long before;
    int b0, b1;
    const long long W = scan_steps(a, g, scan, &before, &b0, &b1);
    const int shares = W > 0 ? share_count(W, blocks, least) : 0;
    const int cut = blockIdx.x + 1;
    if (cut >= shares) return;
    const long long x = share_begin(W, cut, shares);
    const Cursor c = seek(a, g, scan, x, before, b0, b1);
    const long long start = x - c.step, end = start + c.steps;
    if (c.step == 0 || share_begin(W, cut - 1, shares) > start) return;
    int parts = 1;                                                 // share cut - 1 has the first
    while (cut + parts - 1 < shares && share_begin(W, cut + parts - 1, shares) < end) ++parts;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = c.s.n * a.group;
    auto slot = [&](int i) { return i == 0 ? 2 * static_cast<size_t>(cut - 1) + 1 : 2 * static_cast<size_t>(cut - 1 + i); };
    for (int r = blockIdx.y * JN_WARPS + warp; r < g.M; r += gridDim.y * JN_WARPS) {
        const int rr = c.mt * g.M + r;
        if (rr >= rows) break;
        float m = -INFINITY;
        for (int i = lane; i < parts; i += 32) m = fmaxf(m, p.ml[(slot(i) * g.M + r) * 2]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float ref = m == -INFINITY ? 0.f : m;
        float l = 0.f, acc[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) acc[j] = 0.f;
#pragma unroll 4
        for (int i = 0; i < parts; ++i) {
            const size_t at = slot(i) * g.M + r;
            const float2 v = *reinterpret_cast<const float2*>(p.ml + at * 2);
            const float f = exp2f(v.x - ref);
            const float* o = p.o + at * (32 * EPL) + lane * EPL;
            l += v.y * f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) acc[j] += o[j] * f;
        }
        const int i = rr / a.group, head = c.h * a.group + rr % a.group;
        const long long row = c.s.row0 + i;
        const float inv = l == 0.f ? 0.f : a.c.v_scale / l;
        uint32_t w[EPL / 2];
#pragma unroll
        for (int j = 0; j < EPL; j += 2) w[j / 2] = l == 0.f ? 0u : pack_bf16x2(acc[j] * inv, acc[j + 1] * inv);
        uint16_t* dst = a.out + row * a.out_stride + head * (32 * EPL) + lane * EPL;
        if constexpr (EPL == 2) *reinterpret_cast<uint32_t*>(dst) = w[0];
        else if constexpr (EPL == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[EPL / 2 - 2], w[EPL / 2 - 1]);
        if (a.lse != nullptr && lane == 0) a.lse[row * a.n_q + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2F;
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_tiled() {
    static EncodeTiledFn fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return static_cast<EncodeTiledFn>(nullptr);
        return reinterpret_cast<EncodeTiledFn>(ptr);
    }();
    return fn;
}

}  // namespace

// K or V of a cache as (dimension within a 128-byte span, slot, span, kv head, page): a box
// of all spans of box_rows slots of one head lands as [span][slot][128 bytes], swizzled.
// With all_spans false a box is one span.
bool make_kv_map(CUtensorMap* m, const AttnArgs& a, bool v, int box_rows, bool all_spans) {
    EncodeTiledFn fn = encode_tiled();
    if (fn == nullptr) return false;
    const int esz = a.f8 ? 1 : 2;
    const int span = a.head_dim * esz < 128 ? a.head_dim * esz : 128;          // bytes
    const cuuint64_t dims[5] = {static_cast<cuuint64_t>(span / esz), cuuint64_t{1} << a.c.page_shift,
                                static_cast<cuuint64_t>(a.head_dim * esz / span), static_cast<cuuint64_t>(a.c.n_kv),
                                static_cast<cuuint64_t>(a.c.num_pages)};
    // (strides over dimensions of size 1 only have to be valid)
    const cuuint64_t slot = static_cast<cuuint64_t>(a.c.slot_b);
    const cuuint64_t strides[4] = {slot, static_cast<cuuint64_t>(span), a.c.n_kv > 1 ? static_cast<cuuint64_t>(a.c.head_b) : slot,
                                   a.c.num_pages > 1 ? static_cast<cuuint64_t>(a.c.page_b) : slot};
    const cuuint32_t box[5] = {static_cast<cuuint32_t>(span / esz), static_cast<cuuint32_t>(box_rows),
                               all_spans ? static_cast<cuuint32_t>(a.head_dim * esz / span) : 1u, 1, 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return fn(m, a.f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, v ? a.c.v : a.c.k, dims, strides,
              box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, span == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_tree_attn_join(const AttnArgs& a, Tiling g, Partials p, int blocks, int least, cudaStream_t st) {
    if (blocks < 2) return cudaSuccess;
    ProfileScope ps("tree_attention_join", st);
    const dim3 grid(blocks - 1, (g.M + 15) / 16);
    if (a.head_dim == 64) join_kernel<2><<<grid, JN_WARPS * 32, 0, st>>>(a, g, p, blocks, least);
    else if (a.head_dim == 128) join_kernel<4><<<grid, JN_WARPS * 32, 0, st>>>(a, g, p, blocks, least);
    else join_kernel<8><<<grid, JN_WARPS * 32, 0, st>>>(a, g, p, blocks, least);
    note_launch();
    return cudaGetLastError();
}

}  // namespace sre
