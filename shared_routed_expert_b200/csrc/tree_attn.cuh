// Attention over a paged cache: what its kernels share.
#pragma once

#include "kv_cache.cuh"

namespace sre {

struct AttnArgs {
    KvView c;
    int T, n_q, group;                   // group: query heads per kv head
    int head_dim;
    bool f8;
    float scale_log2;                    // softmax_scale * k_scale * log2(e)
    const uint16_t* q;
    long long q_stride;
    const uint64_t* mask;                // null: chain
    int mask_words;
    uint16_t* out;
    long long out_stride;
    float* lse;
    DevStatus* status;
};

// new rows that a sequence may have (rows behind the mask's columns are refused)
__device__ __forceinline__ int attn_max_new(const AttnArgs& a) {
    return a.mask != nullptr ? min(a.c.max_new, 64 * a.mask_words) : a.c.max_new;
}

// whether new token i of a sequence (row t of the call) sees the sequence's new token j
__device__ __forceinline__ bool sees_new(const AttnArgs& a, int t, int i, int j) {
    if (a.mask == nullptr) return j <= i;
    return (a.mask[static_cast<size_t>(t) * a.mask_words + (j >> 6)] >> (j & 63)) & 1;
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2F = 0.6931471805599453f;

// One query row over cache indexes [lo, hi), key by key, by one warp: lane l holds
// dimensions EPL*l .. of q (scaled by scale_log2) and of acc. m, l: running maximum
// (base 2) and sum. A key the row does not see is not read. This is the definition
// itself, used for rows where a value the row does not see holds an infinity or NaN.
template <int EPL, bool F8>
__device__ __forceinline__ void attend_row(const AttnArgs& a, int b, const SeqInfo& s, int i, int kv_head,
                                           const float (&q)[EPL], int lo, int hi, float& m, float& l,
                                           float (&acc)[EPL], int lane) {
    for (int c = lo; c < hi; ++c) {
        if (c >= s.ctx && !sees_new(a, s.row0 + i, i, c - s.ctx)) continue;
        const long long off = slot_offset(a.c, b, c, kv_head);
        if (off < 0) {
            report(a.status, MOE_ERR_DEVICE, b);
            continue;
        }
        float dot = 0.f;
        float v[EPL];
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int d = lane * EPL + j;
            float k;
            if constexpr (F8) {
                k = e4m3_to_f32(reinterpret_cast<const uint8_t*>(a.c.k + off)[d]);
                v[j] = e4m3_to_f32(reinterpret_cast<const uint8_t*>(a.c.v + off)[d]);
            } else {
                k = bf16_to_f32(reinterpret_cast<const uint16_t*>(a.c.k + off)[d]);
                v[j] = bf16_to_f32(reinterpret_cast<const uint16_t*>(a.c.v + off)[d]);
            }
            dot = fmaf(q[j], k, dot);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, o);
        dot *= a.scale_log2;
        const float m2 = dot > m ? dot : m;                        // (a NaN score makes p and l NaN)
        const float ref = m2 == -INFINITY ? 0.f : m2;
        const float alpha = exp2f((m == -INFINITY ? -INFINITY : m - ref));
        const float p = exp2f(dot - ref);
        l = l * alpha + p;
#pragma unroll
        for (int j = 0; j < EPL; ++j) acc[j] = acc[j] * alpha + (p != 0.f ? p * v[j] : 0.f);
        m = m2;
    }
}

cudaError_t launch_tree_attn_rows(const AttnArgs& a, cudaStream_t st);

}  // namespace sre
