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

// Joins the items that a cut between two shares goes through: block x the one that begins
// in share x and does not end there, with M = max m_p: sum_p 2^{m_p - M} (l_p, o_p), in the
// order of the keys. A warp per row. Bound by latency (a few hundred KB out of L2), so it is
// launched early and waits on the device for the kernel before it.
template <int EPL>
__global__ void __launch_bounds__(JN_WARPS * 32) join_kernel(const AttnArgs a, const int M, const Partials p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const JoinItem c = p.items[blockIdx.x];
    const int parts = c.parts;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto slot = [&](int i) { return 2 * static_cast<size_t>(blockIdx.x + i) + (i == 0); };
    for (int r = blockIdx.y * JN_WARPS + warp; parts > 0 && r < M; r += gridDim.y * JN_WARPS) {
        const int rr = c.mt * M + r;
        if (rr >= c.rows) break;
        float m = -INFINITY;
        for (int i = lane; i < parts; i += 32) m = fmaxf(m, p.ml[(slot(i) * M + r) * 2]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const float ref = m == -INFINITY ? 0.f : m;
        float l = 0.f, acc[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) acc[j] = 0.f;
#pragma unroll 8
        for (int i = 0; i < parts; ++i) {
            const size_t at = slot(i) * M + r;
            const float2 v = *reinterpret_cast<const float2*>(p.ml + at * 2);
            const float f = exp2f(v.x - ref);
            const float* o = p.o + at * (32 * EPL) + lane * EPL;
            l += v.y * f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) acc[j] += o[j] * f;
        }
        const int i = rr / a.group, head = c.h * a.group + rr % a.group;
        const long long row = c.row0 + i;
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

size_t partials_bytes(int blocks, int M, int head_dim) {
    return (sizeof(JoinItem) * blocks + 255) / 256 * 256 + static_cast<size_t>(2) * blocks * M * (2 + head_dim) * sizeof(float);
}

Partials partials_at(void* mem, int blocks, int M) {
    Partials p;
    p.items = static_cast<JoinItem*>(mem);
    p.ml = reinterpret_cast<float*>(static_cast<char*>(mem) + (sizeof(JoinItem) * blocks + 255) / 256 * 256);
    p.o = p.ml + static_cast<size_t>(2) * blocks * M * 2;
    return p;
}

cudaError_t launch_tree_attn_join(const AttnArgs& a, int M, Partials p, int blocks, cudaStream_t st) {
    if (blocks < 2) return cudaSuccess;
    ProfileScope ps("tree_attention_join", st);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks - 1, (M + JN_WARPS - 1) / JN_WARPS);
    cfg.blockDim = dim3(JN_WARPS * 32);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const cudaError_t e = a.head_dim == 64    ? cudaLaunchKernelEx(&cfg, join_kernel<2>, a, M, p)
                          : a.head_dim == 128 ? cudaLaunchKernelEx(&cfg, join_kernel<4>, a, M, p)
                                              : cudaLaunchKernelEx(&cfg, join_kernel<8>, a, M, p);
    note_launch();
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace sre
