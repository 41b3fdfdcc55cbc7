// Fused QK-norm + partial RoPE with the append to the paged cache, and the move of
// accepted draft tokens' keys and values inside it.
//
// Append, per token t (sequence b, cache index ctx_len[b] + i) and head:
//   u = v / sqrt(mean(v^2) + eps) * w, the first rot_dim dimensions of u rotated
//   by the table row positions[t] (q and k heads, as in qknorm.cu);
//   q heads -> q_out, k heads -> K cache, v heads unchanged -> V cache.
// Bound by HBM: each head is read and written once. One warp takes HPW
// consecutive heads of a token, lane l holding dimensions EPL*l .. EPL*l + EPL-1,
// all its loads issued before the arithmetic.
#include "kernels.cuh"
#include "kv_cache.cuh"

namespace sre {

namespace {

constexpr int AP_WARPS = 8;

template <int EPL>
struct VecOf;
template <>
struct VecOf<2> { using T = uint32_t; };
template <>
struct VecOf<4> { using T = uint2; };
template <>
struct VecOf<8> { using T = uint4; };

template <int EPL>
__device__ __forceinline__ void widen(const typename VecOf<EPL>::T& v, float (&f)[EPL]) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
    for (int j = 0; j < EPL / 2; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}

// EPL E4M3 codes of f / scale
template <int EPL>
__device__ __forceinline__ void store_e4m3(char* dst, const float (&f)[EPL], float scale) {
    if constexpr (EPL == 2) {
        *reinterpret_cast<uint16_t*>(dst) =
            __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f[0], scale), __fdiv_rn(f[1], scale)), __NV_SATFINITE,
                                     __NV_E4M3);
    } else {
        uint32_t w[EPL / 4];
#pragma unroll
        for (int j = 0; j < EPL / 4; ++j)
            w[j] = pack_e4m3x4(__fdiv_rn(f[4 * j], scale), __fdiv_rn(f[4 * j + 1], scale),
                               __fdiv_rn(f[4 * j + 2], scale), __fdiv_rn(f[4 * j + 3], scale));
        if constexpr (EPL == 4) *reinterpret_cast<uint32_t*>(dst) = w[0];
        else *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[EPL / 4 - 1]);
    }
}

struct AppendArgs {
    int T, n_q, rot, max_pos;
    float eps;
    const uint16_t* qkv;                 // may be q_out (in place)
    long long qkv_stride, q_stride;
    const int32_t* pos;
    const uint16_t* q_w;
    const uint16_t* k_w;
    const float* cos_sin;
    uint16_t* q_out;
    int32_t* bad;
};

template <int EPL, int HPW, bool F8>
__global__ void __launch_bounds__(AP_WARPS * 32) append_kernel(const AppendArgs a, const KvView c) {
    constexpr int D = 32 * EPL;
    using V = typename VecOf<EPL>::T;
    const int lane = threadIdx.x & 31;
    const int heads = a.n_q + 2 * c.n_kv;
    const int groups = (heads + HPW - 1) / HPW;
    const long long item = static_cast<long long>(blockIdx.x) * AP_WARPS + (threadIdx.x >> 5);
    if (item >= static_cast<long long>(a.T) * groups) return;
    const int t = static_cast<int>(item / groups);
    const int h0 = static_cast<int>(item % groups) * HPW;
    const int nh = min(HPW, heads - h0);

    // the loads of the rows do not wait for the checks: every row t < T exists
    const V* in = reinterpret_cast<const V*>(a.qkv + t * a.qkv_stride + static_cast<long long>(h0) * D);
    V raw[HPW];
#pragma unroll
    for (int k = 0; k < HPW; ++k)
        if (k < nh) raw[k] = in[k * 32 + lane];

    const int b = seq_of_row(c.q_start, c.B, t, lane);
    if (b < 0 || t >= c.q_start[b + 1]) return;                    // padding
    const bool counts = h0 <= a.n_q && a.n_q < h0 + nh;            // this warp has the first k head
    int p = 0;
    if (a.rot > 0) {
        p = a.pos[t];
        if (p < 0 || p >= a.max_pos) {
            if (counts && lane == 0 && a.bad != nullptr) atomicAdd(a.bad, 1);
            return;
        }
    }
    long long slot = -1;
    if (h0 + nh > a.n_q) {
        const SeqInfo s = seq_info(c, b, a.T, c.max_new);
        if (s.ok) slot = slot_offset(c, b, s.ctx + (t - s.row0), 0);
        if (slot < 0 && counts && lane == 0 && a.bad != nullptr) atomicAdd(a.bad, 1);
    }

    const int half = a.rot >> 1;
    const int i0 = lane * EPL;                 // first dimension of this lane
    const int lane_off = half / EPL;           // rotation partners are this many lanes apart
    const int src = (i0 < half) ? lane + lane_off : (i0 < a.rot ? lane - lane_off : lane);
    float co[EPL], sn[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        co[j] = 1.0f;
        sn[j] = 0.0f;
    }
    if (i0 < a.rot && h0 < a.n_q + c.n_kv) {
        const float* cs = a.cos_sin + static_cast<long long>(p) * a.rot + (i0 < half ? i0 : i0 - half);
        const float sign = i0 < half ? -1.0f : 1.0f;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            co[j] = cs[j];
            sn[j] = sign * cs[half + j];
        }
    }
    float wq[EPL], wk[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) wq[j] = wk[j] = 1.0f;
    if (a.q_w != nullptr && h0 < a.n_q) widen<EPL>(reinterpret_cast<const V*>(a.q_w)[lane], wq);
    if (a.k_w != nullptr && h0 + nh > a.n_q) widen<EPL>(reinterpret_cast<const V*>(a.k_w)[lane], wk);

#pragma unroll
    for (int k = 0; k < HPW; ++k) {
        if (k >= nh) break;                                        // warp-uniform
        const int h = h0 + k;
        if (h >= a.n_q + c.n_kv) {                                 // a v head
            if (slot < 0) continue;
            char* dst = c.v + slot + (h - a.n_q - c.n_kv) * c.head_b;
            if constexpr (F8) {
                float v[EPL];
                widen<EPL>(raw[k], v);
                store_e4m3<EPL>(dst + lane * EPL, v, c.v_scale);
            } else {
                reinterpret_cast<V*>(dst)[lane] = raw[k];
            }
            continue;
        }
        const bool is_q = h < a.n_q;
        if (!is_q && slot < 0) continue;
        float v[EPL];
        widen<EPL>(raw[k], v);
        const bool norm = (is_q ? a.q_w : a.k_w) != nullptr;
        float r = 1.0f;
        if (norm) {
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < EPL; ++j) ss = fmaf(v[j], v[j], ss);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, off);
            r = rsqrtf(ss / D + a.eps);
        }
        float y[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const float u = v[j] * r * (is_q ? wq[j] : wk[j]);
            const float partner = __shfl_sync(0xFFFFFFFFu, u, src);
            // dimensions that do not rotate pass through whatever their value (0 * infinity)
            y[j] = i0 < a.rot ? u * co[j] + partner * sn[j] : u;
        }
        if (!is_q && F8) {
            store_e4m3<EPL>(c.k + slot + (h - a.n_q) * c.head_b + lane * EPL, y, c.k_scale);
        } else {
            uint32_t o[EPL / 2];
#pragma unroll
            for (int j = 0; j < EPL; j += 2) o[j >> 1] = pack_bf16x2(y[j], y[j + 1]);
            V* dst = is_q ? reinterpret_cast<V*>(a.q_out + t * a.q_stride + static_cast<long long>(h) * D)
                          : reinterpret_cast<V*>(c.k + slot + (h - a.n_q) * c.head_b);
            dst[lane] = *reinterpret_cast<const V*>(o);
        }
    }
}

template <int EPL>
void append_epl(const AppendArgs& a, const KvView& c, bool f8, cudaStream_t st) {
    constexpr int HPW = 8;
    const long long items = static_cast<long long>(a.T) * ((a.n_q + 2 * c.n_kv + HPW - 1) / HPW);
    const unsigned blocks = static_cast<unsigned>((items + AP_WARPS - 1) / AP_WARPS);
    if (f8) append_kernel<EPL, HPW, true><<<blocks, AP_WARPS * 32, 0, st>>>(a, c);
    else append_kernel<EPL, HPW, false><<<blocks, AP_WARPS * 32, 0, st>>>(a, c);
}

// Compaction. A thread owns one 16-byte column of one (layer, K or V, head) of a
// sequence and walks the accepted tokens in ascending order: sources never lie in
// front of their destinations and nobody else touches its column, so reading a few
// tokens ahead of the writes keeps the move in place and free of barriers.
constexpr int CP_THREADS = 256;
constexpr int CP_AHEAD = 8;

__global__ void __launch_bounds__(CP_THREADS) compact_kernel(const KvView c, int n_layers, long long layer_b,
                                                             const int32_t* __restrict__ accepted, int max_accept,
                                                             const int32_t* __restrict__ n_accepted, int row_chunks,
                                                             int32_t* bad) {
    extern __shared__ long long cp_off[];                          // [2][n] source and destination byte offsets
    const int b = blockIdx.y;
    const int n = n_accepted[b];
    const long long new_n = static_cast<long long>(c.q_start[b + 1]) - c.q_start[b];
    const int ctx = c.ctx_len[b];
    bool ok = n >= 0 && n <= max_accept && new_n >= 0 && new_n <= c.max_new && ctx >= 0 &&
              ctx + new_n <= (static_cast<long long>(c.max_pages) << c.page_shift);
    if (ok) {
        for (int i = threadIdx.x; i < n; i += CP_THREADS) {
            const int at = accepted[static_cast<long long>(b) * max_accept + i];
            const int before = i > 0 ? accepted[static_cast<long long>(b) * max_accept + i - 1] : -1;
            if (at <= before || at < 0 || at >= new_n) {           // (at >= i follows from the order)
                ok = false;
                break;
            }
            const long long s = slot_offset(c, b, ctx + at, 0), d = slot_offset(c, b, ctx + i, 0);
            if (s < 0 || d < 0) {
                ok = false;
                break;
            }
            cp_off[i] = s;
            cp_off[max_accept + i] = d;
        }
    }
    if (!__syncthreads_and(ok)) {
        if (blockIdx.x == 0 && threadIdx.x == 0 && bad != nullptr) atomicAdd(bad, 1);
        return;
    }
    const long long cols = static_cast<long long>(n_layers) * 2 * c.n_kv * row_chunks;
    const long long col = static_cast<long long>(blockIdx.x) * CP_THREADS + threadIdx.x;
    if (col >= cols) return;
    const int chunk = static_cast<int>(col % row_chunks);
    long long rest = col / row_chunks;
    const int h = static_cast<int>(rest % c.n_kv);
    rest /= c.n_kv;
    char* base = ((rest & 1) ? c.v : c.k) + (rest >> 1) * layer_b + h * c.head_b + chunk * 16;
    for (int i0 = 0; i0 < n; i0 += CP_AHEAD) {
        uint4 x[CP_AHEAD];
#pragma unroll
        for (int j = 0; j < CP_AHEAD; ++j) {
            const int i = i0 + j;
            if (i < n && cp_off[i] != cp_off[max_accept + i]) x[j] = *reinterpret_cast<const uint4*>(base + cp_off[i]);
        }
#pragma unroll
        for (int j = 0; j < CP_AHEAD; ++j) {
            const int i = i0 + j;
            if (i < n && cp_off[i] != cp_off[max_accept + i])
                *reinterpret_cast<uint4*>(base + cp_off[max_accept + i]) = x[j];
        }
    }
}

}  // namespace

cudaError_t launch_append(const KvView& c, int head_dim, bool f8, int T, int n_q, int rot, float eps, const uint16_t* qkv,
                          long long qkv_stride, const int32_t* pos, int max_pos, const uint16_t* q_w, const uint16_t* k_w,
                          const float* cos_sin, uint16_t* q_out, long long q_stride, int32_t* bad, cudaStream_t st) {
    ProfileScope ps("qk_norm_rope_append", st);
    AppendArgs a{T, n_q, rot, max_pos, eps, qkv, qkv_stride, q_stride, pos, q_w, k_w, cos_sin, q_out, bad};
    if (head_dim == 64) append_epl<2>(a, c, f8, st);
    else if (head_dim == 128) append_epl<4>(a, c, f8, st);
    else append_epl<8>(a, c, f8, st);
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_compact(const KvView& c, int row_bytes, int n_layers, long long layer_b, const int32_t* accepted,
                           int max_accept, const int32_t* n_accepted, int32_t* bad, cudaStream_t st) {
    ProfileScope ps("kv_compact", st);
    const int row_chunks = row_bytes / 16;
    const long long cols = static_cast<long long>(n_layers) * 2 * c.n_kv * row_chunks;
    const dim3 grid(static_cast<unsigned>((cols + CP_THREADS - 1) / CP_THREADS), c.B);
    compact_kernel<<<grid, CP_THREADS, 2 * sizeof(long long) * max_accept, st>>>(c, n_layers, layer_b, accepted,
                                                                                 max_accept, n_accepted, row_chunks, bad);
    note_launch();
    return cudaGetLastError();
}

}  // namespace sre
