// Fused QK-norm + partial RoPE with the append to the paged cache, and the move of
// accepted draft tokens' keys and values inside it.
//
// Append, per token t (sequence b, cache index ctx_len[b] + i) and head:
//   u = v / sqrt(mean(v^2) + eps) * w, the first rot_dim dimensions of u rotated
//   by the table row positions[t] (q and k heads, as in qknorm.cu);
//   q heads -> q_out, k heads -> K cache, v heads unchanged -> V cache.
// Each head is read and written once; what the kernel spends beside that is instructions, so
// lanes hold 8 dimensions each (16-byte loads and stores) and a warp's instruction covers 1, 2
// or 4 heads of 256, 128 or 64 dimensions. The sums of squares are added in the order of
// qknorm.cu's 32 lanes (partial sums of head_dim / 32 dimensions, a butterfly over them), and
// the products are formed alike, so q rows and bf16 keys have the same bits. 5 prompts of 5949
// tokens, 96 + 8 + 8 heads of 128, 340 MB: 78 us, 4.4 TB/s; the warps wait on their loads and
// butterflies (4 dimensions a lane and a head per instruction: 104 instructions a head, 86 us).
#include "kernels.cuh"
#include "kv_cache.cuh"

namespace sre {

namespace {

constexpr int AP_WARPS = 8;

__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
}

template <int N>
struct Floats;
template <>
struct Floats<2> {
    using T = float2;
    static __device__ __forceinline__ float2 of(float v) { return make_float2(v, v); }
};
template <>
struct Floats<4> {
    using T = float4;
    static __device__ __forceinline__ float4 of(float v) { return make_float4(v, v, v, v); }
};

// 8 E4M3 codes of f / scale
__device__ __forceinline__ uint2 codes8(const float (&f)[8], float scale) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __fdiv_rn(f[j], scale);
    return make_uint2(pack_e4m3x4(q[0], q[1], q[2], q[3]), pack_e4m3x4(q[4], q[5], q[6], q[7]));
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

// LPH lanes per head; SH: half of rot modulo 8 (how far a dimension's rotation partner lies from it
// among a lane's 8); KI: instructions' worth of heads per warp.
template <int LPH, int SH, int KI, bool F8>
__global__ void __launch_bounds__(AP_WARPS * 32, 4) append_kernel(const AppendArgs a, const KvView c) {
    constexpr int D = 8 * LPH, HPI = 32 / LPH, HPW = KI * HPI;
    constexpr int PS = D / 32, NP = 8 / PS;                        // dimensions per partial sum, partial sums per lane
    const int lane = threadIdx.x & 31, L = lane % LPH, sub = lane / LPH;
    const int heads = a.n_q + 2 * c.n_kv;
    const int groups = (heads + HPW - 1) / HPW;
    const long long item = static_cast<long long>(blockIdx.x) * AP_WARPS + (threadIdx.x >> 5);
    if (item >= static_cast<long long>(a.T) * groups) return;
    const int t = static_cast<int>(item / groups);
    const int h0 = static_cast<int>(item % groups) * HPW;
    const int nh = min(HPW, heads - h0);

    // the loads of the rows do not wait for the checks: every row t < T exists
    const uint16_t* in = a.qkv + t * a.qkv_stride + static_cast<long long>(h0 + sub) * D + L * 8;
    uint4 raw[KI];
#pragma unroll
    for (int k = 0; k < KI; ++k)
        if (k * HPI + sub < nh) raw[k] = *reinterpret_cast<const uint4*>(in + k * HPI * D);
    const int p = a.rot > 0 ? a.pos[t] : 0;

    const int b = seq_of_row(c.q_start, c.B, t, lane);
    if (b < 0 || t >= c.q_start[b + 1]) return;                    // padding
    const bool counts = h0 <= a.n_q && a.n_q < h0 + nh;            // this warp has the first k head
    if (a.rot > 0 && (p < 0 || p >= a.max_pos)) {
        if (counts && lane == 0 && a.bad != nullptr) atomicAdd(a.bad, 1);
        return;
    }
    const int i0 = L * 8, half = a.rot >> 1;   // first dimension of this lane
    const float* cs = a.cos_sin + static_cast<long long>(p) * a.rot;
    float co[8], sn[8];
#pragma unroll
    for (int n = 0; n < NP; ++n) {             // PS dimensions rotate alike
        const int d = i0 + n * PS;
        const bool turn = d < a.rot && h0 < a.n_q + c.n_kv;
        const int at = d < half ? d : d - half;
        const float sign = d < half ? -1.0f : 1.0f;
        using F = typename Floats<PS < 4 ? 2 : 4>::T;
#pragma unroll
        for (int j = 0; j < PS; j += (PS < 4 ? 2 : 4)) {
            F x = Floats<PS < 4 ? 2 : 4>::of(1.0f), y = Floats<PS < 4 ? 2 : 4>::of(0.0f);
            if (turn) {
                x = *reinterpret_cast<const F*>(cs + at + j);
                y = *reinterpret_cast<const F*>(cs + half + at + j);
            }
#pragma unroll
            for (int e = 0; e < (PS < 4 ? 2 : 4); ++e) {
                co[n * PS + j + e] = reinterpret_cast<const float*>(&x)[e];
                sn[n * PS + j + e] = sign * reinterpret_cast<const float*>(&y)[e];
            }
        }
    }
    long long slot = -1;
    if (h0 + nh > a.n_q) {
        const SeqInfo s = seq_info(c, b, a.T, c.max_new);
        if (s.ok && t >= s.row0) slot = slot_offset(c, b, s.ctx + (t - s.row0), 0);   // (q_start out of order: not followed)
        if (slot < 0 && counts && lane == 0 && a.bad != nullptr) atomicAdd(a.bad, 1);
    }
    // norm weights as they are stored (registers decide how many warps are in flight)
    uint4 wq = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u), wk = wq;   // 1.0
    if (a.q_w != nullptr && h0 < a.n_q) wq = reinterpret_cast<const uint4*>(a.q_w)[L];
    if (a.k_w != nullptr && h0 + nh > a.n_q) wk = reinterpret_cast<const uint4*>(a.k_w)[L];
    // dimension d's partner is d + half in the first half and d - half in the second
    int src[NP];
    bool turns[NP];
#pragma unroll
    for (int n = 0; n < NP; ++n) {
        const int d = i0 + n * PS;
        turns[n] = d < a.rot;
        src[n] = sub * LPH + (d < half ? (d + half) >> 3 : (turns[n] ? (d - half) >> 3 : L));
    }

    // u = v r w of 8 dimensions, r from the head's mean square
    auto normed = [&](const float (&v)[8], const float (&w)[8], bool norm, float (&u)[8]) {
        float ss[NP];
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            ss[n] = 0.0f;
#pragma unroll
            for (int j = 0; j < PS; ++j) ss[n] = fmaf(v[n * PS + j], v[n * PS + j], ss[n]);
        }
#pragma unroll
        for (int off = LPH / 2; off > 0; off >>= 1)
#pragma unroll
            for (int n = 0; n < NP; ++n) ss[n] += __shfl_xor_sync(0xFFFFFFFFu, ss[n], off);
#pragma unroll
        for (int off = NP / 2; off > 0; off >>= 1)
#pragma unroll
            for (int n = 0; n < off; ++n) ss[n] += ss[n + off];
        const float r = norm ? rsqrtf(ss[0] / D + a.eps) : 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = v[j] * r * w[j];
    };
    // every lane offers the element its taker is after: (j + SH) % 8 to a taker in the first half of the
    // rotating dimensions, (j - SH) % 8 to one in the second
    auto partner = [&](const float (&u)[8], int j) {
        const float o = __shfl_sync(0xFFFFFFFFu, u[(j + SH) & 7], src[j / PS]);
        if constexpr (SH % 4 == 0) return o;
        const float p2 = __shfl_sync(0xFFFFFFFFu, u[(j - SH) & 7], src[j / PS]);
        return i0 + j < half ? o : p2;
    };

    if (h0 + HPW <= a.n_q && a.q_w != nullptr) {
        // q heads alone (most warps): nothing to tell apart
        float w[8];
        widen8(wq, w);
        uint16_t* dst = a.q_out + t * a.q_stride + static_cast<long long>(h0 + sub) * D + i0;
#pragma unroll
        for (int k = 0; k < KI; ++k) {
            float v[8], u[8], y[8];
            widen8(raw[k], v);
            normed(v, w, true, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float o = partner(u, j);
                // dimensions that do not rotate pass through whatever their value and that of what is offered
                // to them, another dimension if SH is not 0 (0 * infinity; 0.7% of a prompt's time)
                y[j] = turns[j / PS] ? u[j] * co[j] + o * sn[j] : u[j];
            }
            *reinterpret_cast<uint4*>(dst + k * HPI * D) =
                make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
        }
        return;
    }
#pragma unroll 1
    for (int k = 0; k < KI; ++k) {
        const int h = h0 + k * HPI + sub;
        if (k * HPI >= nh) break;                                  // warp-uniform
        const bool is_q = h < a.n_q, is_v = h >= a.n_q + c.n_kv, real = h < heads;
        uint4 x = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int q = 0; q < KI; ++q)
            if (q == k && real) x = raw[q];
        float v[8], u[8], y[8], w[8];
        widen8(x, v);
        widen8(is_q ? wq : wk, w);
        // (all lanes take part in the shuffles, whatever their heads)
        normed(v, w, (is_q ? a.q_w : a.k_w) != nullptr, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float o = partner(u, j);
            y[j] = turns[j / PS] ? u[j] * co[j] + o * sn[j] : u[j];
        }
        if (!real || (!is_q && slot < 0)) continue;
        const uint4 out = is_v ? x
                               : make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                                            pack_bf16x2(y[6], y[7]));
        if (is_q) {
            *reinterpret_cast<uint4*>(a.q_out + t * a.q_stride + static_cast<long long>(h) * D + i0) = out;
            continue;
        }
        char* dst = (is_v ? c.v + (h - a.n_q - c.n_kv) * c.head_b : c.k + (h - a.n_q) * c.head_b) + slot;
        if constexpr (F8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = is_v ? v[j] : y[j];
            *reinterpret_cast<uint2*>(dst + i0) = codes8(y, is_v ? c.v_scale : c.k_scale);
        } else {
            *reinterpret_cast<uint4*>(dst + i0 * 2) = out;
        }
    }
}

template <int LPH, int SH, int KI>
void append_ki(const AppendArgs& a, const KvView& c, bool f8, cudaStream_t st) {
    constexpr int HPW = KI * (32 / LPH);
    const long long items = static_cast<long long>(a.T) * ((a.n_q + 2 * c.n_kv + HPW - 1) / HPW);
    const unsigned blocks = static_cast<unsigned>((items + AP_WARPS - 1) / AP_WARPS);
    if (f8) append_kernel<LPH, SH, KI, true><<<blocks, AP_WARPS * 32, 0, st>>>(a, c);
    else append_kernel<LPH, SH, KI, false><<<blocks, AP_WARPS * 32, 0, st>>>(a, c);
}

template <int LPH, int SH>
void append_sh(const AppendArgs& a, const KvView& c, bool f8, cudaStream_t st) {
    // 4 instructions' worth of heads a warp: 16, 8 or 4 of 64, 128 or 256 dimensions (of 256, 3000 tokens of
    // 112 heads: 73 us, with 8 heads a warp 82, with 2 88)
    constexpr int KI = 4;
    // a decode batch that the SMs hold at once takes half as many heads a warp: a shorter chain
    // (1 token of 112 heads 2.9 against 3.4 us, 64 tokens 4.1 against 4.8 us), while more heads
    // share what is looked up per token in a prefill chunk (5949 tokens 78 against 100 us)
    if (static_cast<long long>(a.T) * (a.n_q + 2 * c.n_kv) <= 16384) append_ki<LPH, SH, KI / 2>(a, c, f8, st);
    else append_ki<LPH, SH, KI>(a, c, f8, st);
}

// Compaction. A thread owns one 16-byte column of one (layer, K or V, head) of a
// sequence and walks the accepted tokens in ascending order: sources never lie in
// front of their destinations and nobody else touches its column, so reading a few
// tokens ahead of the writes keeps the move in place and free of barriers. Rows of 64 to 512
// bytes here and there, bound by their latency: 92 layers of 8 heads of 128 E4M3, 32 sequences,
// 60 MB, 16.5 us (two columns a thread 17.4, four 20.3).
constexpr int CP_THREADS = 256;
constexpr int CP_AHEAD = 8;              // tokens read before the first of them is written

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
    const int sh = (rot / 2) % 8;              // a multiple of head_dim / 32
    if (head_dim == 256) append_sh<32, 0>(a, c, f8, st);
    else if (head_dim == 128) sh == 0 ? append_sh<16, 0>(a, c, f8, st) : append_sh<16, 4>(a, c, f8, st);
    else if (sh == 0) append_sh<8, 0>(a, c, f8, st);
    else if (sh == 2) append_sh<8, 2>(a, c, f8, st);
    else if (sh == 4) append_sh<8, 4>(a, c, f8, st);
    else append_sh<8, 6>(a, c, f8, st);
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
