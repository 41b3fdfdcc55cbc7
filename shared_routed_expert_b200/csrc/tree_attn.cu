// Attention of new tokens (decode rows, drafted chains and trees, prefill chunks)
// over a paged cache:
//   s_j = softmax_scale * q . k_j over the keys a row sees, m = max s, p_j = e^{s_j - m},
//   out = sum p_j v_j / sum p_j,  lse = m + ln sum p_j.
// Here: the join of partial results, and the cache's TMA maps.
#include <atomic>

#include "kernels.cuh"
#include "tree_attn.cuh"

namespace sre {

namespace {

constexpr int JN_WARPS = 4;
std::atomic<int> g_stall{0};

// Joins the items that a cut between two shares goes through: block x the one that begins
// in share x and does not end there; a warp takes every 16th row. Bound by latency and L2
// (some tens of MB). Its launch is hidden behind the kernel before it, whose blocks have all ended
// when it starts (none of them lets it start sooner) and whose results it waits for on the device
// (13 of 185 us for trees of up to 61 nodes; 4-token chains with a block per 4 rows 113 us, per
// 16 rows 108 us, with 8 parts' loads in flight instead of 4 109 us).
template <int EPL>
__global__ void __launch_bounds__(JN_WARPS * 32) join_kernel(const AttnArgs a, const int M, const Partials p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const JoinItem c = p.items[blockIdx.x];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int r = blockIdx.y * JN_WARPS + warp; c.parts > 0 && r < M && c.mt * M + r < c.rows; r += gridDim.y * JN_WARPS)
        join_row<EPL, 4>(a, p, M, blockIdx.x, c.parts, c.row0, c.h, r, c.mt * M + r, lane);
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

void tree_attn_inject_stall(int n_calls) { g_stall.store(n_calls); }

bool tree_attn_take_stall() {
    int n = g_stall.load();
    while (n > 0)
        if (g_stall.compare_exchange_weak(n, n - 1)) return true;
    return false;
}

long long tile_wait_limit(const AttnArgs& a) {
    const long long keys = static_cast<long long>(a.c.max_pages) << a.c.page_shift, most = 1ll << 22;
    return (16ll << 30) + (keys < most ? keys : most) * 32 * 8192;
}

// K or V of a cache as (dimension within a 128-byte span, slot, span, kv head, page): a box
// is one span of box_rows slots of one head, stored [slot][128 bytes] (64 for 64-byte
// rows) with the swizzle of that width.
bool make_kv_map(CUtensorMap* m, const AttnArgs& a, bool v, int box_rows) {
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
                               1, 1, 1};
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return fn(m, a.f8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, v ? a.c.v : a.c.k, dims, strides,
              box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, span == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// the counters come first, at one place whatever the kernel, so that they stay zero between calls
constexpr size_t kCounterBytes = 2048;
static_assert(kCounterBytes >= kSmallBlocks * sizeof(unsigned) && kCounterBytes >= kTileBlocks * sizeof(unsigned), "a counter per block");

size_t partials_bytes(int blocks, int M, int head_dim) {
    return kCounterBytes + (sizeof(JoinItem) * blocks + 255) / 256 * 256 +
           static_cast<size_t>(2) * blocks * M * (2 + head_dim) * sizeof(float);
}

Partials partials_at(void* mem, int blocks, int M) {
    Partials p;
    char* at = static_cast<char*>(mem);
    p.arrived = reinterpret_cast<unsigned*>(at);
    p.items = reinterpret_cast<JoinItem*>(at + kCounterBytes);
    p.ml = reinterpret_cast<float*>(at + kCounterBytes + (sizeof(JoinItem) * blocks + 255) / 256 * 256);
    p.o = p.ml + static_cast<size_t>(2) * blocks * M * 2;
    return p;
}

cudaError_t launch_tree_attn_join(const AttnArgs& a, int M, Partials p, int blocks, cudaStream_t st) {
    if (blocks < 2) return cudaSuccess;
    ProfileScope ps("tree_attention_join", st);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks - 1, (M + 4 * JN_WARPS - 1) / (4 * JN_WARPS));
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
