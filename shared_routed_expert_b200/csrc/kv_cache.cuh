// Paged key/value cache: what the append, attention and compaction kernels share.
#pragma once

#include "common.cuh"

namespace sre {

constexpr int kMaxSeqs = 4096;           // sequences of one call

// One layer's cache with byte strides, and the sequences of a call, as the kernels take them.
struct KvView {
    char* k;
    char* v;
    long long page_b, head_b, slot_b;    // byte strides
    int num_pages, page_shift, n_kv;
    float k_scale, v_scale;
    const int32_t* q_start;
    const int32_t* ctx_len;
    const int32_t* page_table;
    int B, max_pages, max_new;
};

struct SeqInfo {
    int row0, n, ctx;                    // first row, new rows, cached tokens
    bool ok;                             // false: contents out of range (n is 0 then)
};

// Sequence b's rows and lengths, checked against T rows, max_new (and max_n, the
// mask's columns) and the page table's width.
__device__ __forceinline__ SeqInfo seq_info(const KvView& c, int b, long long T, int max_n) {
    SeqInfo s;
    s.row0 = c.q_start[b];
    const long long n = static_cast<long long>(c.q_start[b + 1]) - s.row0;
    s.ctx = c.ctx_len[b];
    s.ok = s.row0 >= 0 && n >= 0 && s.row0 + n <= T && n <= max_n && s.ctx >= 0 &&
           s.ctx + n <= (static_cast<long long>(c.max_pages) << c.page_shift);
    s.n = s.ok ? static_cast<int>(n) : 0;
    return s;
}

// Byte offset of (sequence b, cache index idx, kv head h) in K and V, or -1 for a
// page id outside the cache. idx must lie inside the page table's row.
__device__ __forceinline__ long long slot_offset(const KvView& c, int b, int idx, int h) {
    const int page = c.page_table[static_cast<size_t>(b) * c.max_pages + (idx >> c.page_shift)];
    if (page < 0 || page >= c.num_pages) return -1;
    return page * c.page_b + h * c.head_b + (idx & ((1 << c.page_shift) - 1)) * c.slot_b;
}

// The sequence whose rows hold row t: the last b with q_start[b] <= t, for
// ascending q_start; every lane of the warp gets it. -1 in front of the first row.
// A 32-way search: one load per lane and level (3 levels for 4096 sequences).
__device__ __forceinline__ int seq_of_row(const int32_t* q_start, int B, int t, int lane) {
    int lo = 0, n = B;                   // the answer + 1 lies in lo .. lo + n
    while (n > 32) {
        const int step = (n + 31) >> 5;
        const int i = lo + (lane + 1) * step - 1;
        const bool le = i < lo + n && q_start[i] <= t;
        const int k = __popc(__ballot_sync(0xFFFFFFFFu, le));
        const int lo2 = lo + k * step;
        n = min(step, lo + n - lo2);
        lo = lo2;
    }
    const bool le = lane < n && q_start[lo + lane] <= t;
    return lo + __popc(__ballot_sync(0xFFFFFFFFu, le)) - 1;
}

// E4M3 codes of four values (round to nearest even, saturating at 448; NaN stays NaN)
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// four E4M3 codes -> four fp16 (exact)
__device__ __forceinline__ uint2 e4m3x4_to_f16x4(uint32_t v) {
    uint2 r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(r.x), "=r"(r.y)
        : "r"(v));
    return r;
}

}  // namespace sre
