// Attention over a paged cache: what its kernels share.
#pragma once

#include <cuda.h>

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
        for (int j = 0; j < EPL; ++j) acc[j] = acc[j] * alpha + p * v[j];
        m = m2;
    }
}

// ---- splitting the work
// An item is (sequence, kv head, tile of M query rows); the rows of a kv head are
// packed token-major, row r being token r / group, query head r % group. An item takes
// steps of SK keys up to the last key that one of its rows may see. The steps of all
// items, in the order sequence, head, tile, are one axis that is cut into equal shares,
// one per block, so the load is even whatever the lengths; an item that a cut goes
// through leaves partial results (unnormalised sums with their maximum) that are joined
// afterwards in the order of the keys.

struct Tiling {
    int M, SK;
};

// last cache index + 1 that rows of tile mt may see
__device__ __forceinline__ int tile_keys(const AttnArgs& a, const SeqInfo& s, int mt, int M) {
    if (a.mask != nullptr) return s.ctx + s.n;
    const int last = min((mt + 1) * M, s.n * a.group) - 1;
    return s.ctx + last / a.group + 1;
}
__device__ __forceinline__ int tile_steps(const AttnArgs& a, const SeqInfo& s, int mt, Tiling g) {
    return (tile_keys(a, s, mt, g.M) + g.SK - 1) / g.SK;
}
__device__ __forceinline__ int seq_tiles(const AttnArgs& a, const SeqInfo& s, int M) {
    return (s.n * a.group + M - 1) / M;
}
// steps of one kv head of a sequence
__device__ __forceinline__ long long head_steps(const AttnArgs& a, const SeqInfo& s, Tiling g) {
    const int tiles = seq_tiles(a, s, g.M);
    if (tiles == 0) return 0;
    const int lo = tile_steps(a, s, 0, g), hi = tile_steps(a, s, tiles - 1, g);
    if (lo == hi) return static_cast<long long>(tiles) * lo;
    long long sum = 0;
    for (int mt = 0; mt < tiles; ++mt) sum += tile_steps(a, s, mt, g);
    return sum;
}

struct ScanShared {
    long long warp_sum[32];
    long long rem;
    int b;
};

// Number of blocks that share W steps: no more than `blocks`, and no share below
// `least` steps.
__device__ __forceinline__ int share_count(long long W, int blocks, int least) {
    const long long n = (W + least - 1) / least;
    return static_cast<int>(n < blocks ? (n > 1 ? n : 1) : blocks);
}
__device__ __forceinline__ long long share_begin(long long W, int i, int count) { return W * i / count; }

// All steps of the call (W); called by every thread of the block. *before: steps in
// front of this thread's sequences.
__device__ __forceinline__ long long scan_steps(const AttnArgs& a, Tiling g, ScanShared& sh, long long* before, int* b0,
                                                int* b1) {
    const int per = (a.c.B + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    *b0 = min(a.c.B, static_cast<int>(threadIdx.x) * per);
    *b1 = min(a.c.B, *b0 + per);
    long long mine = 0;
    for (int b = *b0; b < *b1; ++b) {
        const SeqInfo s = seq_info(a.c, b, a.T, attn_max_new(a));
        if (!s.ok && blockIdx.x == 0 && blockIdx.y == 0) report(a.status, MOE_ERR_DEVICE, b);
        mine += head_steps(a, s, g) * a.c.n_kv;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += v;
    }
    if (lane == 31) sh.warp_sum[warp] = inc;
    __syncthreads();
    long long base = 0, W = 0;
    for (int w = 0; w < warps; ++w) {
        if (w < warp) base += sh.warp_sum[w];
        W += sh.warp_sum[w];
    }
    *before = base + inc - mine;
    return W;
}

// A place on the axis: an item and the step within it.
struct Cursor {
    SeqInfo s;
    int b, h, mt, step, steps;           // steps: of the whole item

    __device__ __forceinline__ void open(const AttnArgs& a, Tiling g) { steps = tile_steps(a, s, mt, g); }
    // to the first step of the next item (sequences without steps are passed over)
    __device__ __forceinline__ void next(const AttnArgs& a, Tiling g) {
        step = 0;
        if (++mt >= seq_tiles(a, s, g.M)) {
            mt = 0;
            if (++h >= a.c.n_kv) {
                h = 0;
                do {
                    ++b;
                    if (b >= a.c.B) return;
                    s = seq_info(a.c, b, a.T, attn_max_new(a));
                } while (s.n == 0);
            }
        }
        open(a, g);
    }
};

// The place of step x (0 <= x < W), by every thread of the block, after scan_steps.
__device__ __forceinline__ Cursor seek(const AttnArgs& a, Tiling g, ScanShared& sh, long long x, long long before, int b0,
                                       int b1) {
    if (x >= before) {
        long long rem = x - before;
        for (int b = b0; b < b1; ++b) {
            const long long n = head_steps(a, seq_info(a.c, b, a.T, attn_max_new(a)), g) * a.c.n_kv;
            if (rem < n) {
                sh.b = b;
                sh.rem = rem;
                break;
            }
            rem -= n;
        }
    }
    __syncthreads();
    Cursor c;
    c.b = sh.b;
    c.s = seq_info(a.c, c.b, a.T, attn_max_new(a));
    const long long per = head_steps(a, c.s, g);
    c.h = static_cast<int>(sh.rem / per);
    long long rem = sh.rem % per;
    c.mt = 0;
    c.open(a, g);
    if (per == static_cast<long long>(c.steps) * seq_tiles(a, c.s, g.M)) {
        c.mt = static_cast<int>(rem / c.steps);
        rem %= c.steps;
    } else {
        while (rem >= c.steps) {
            rem -= c.steps;
            ++c.mt;
            c.open(a, g);
        }
    }
    c.step = static_cast<int>(rem);
    return c;
}

// Keys c0 .. c0 + 31 that row (token i) of a sequence sees, as bits, of those below `end`
__device__ __forceinline__ uint32_t seen_bits(const AttnArgs& a, const SeqInfo& s, int i, int c0, int end) {
    uint32_t bits = 0xFFFFFFFFu;
    const int j0 = c0 - s.ctx;                                     // new token of bit 0 (< 0: in the prefix)
    if (j0 + 31 >= 0) {
        if (a.mask == nullptr) {
            const int n = i - j0 + 1;                              // visible keys from bit 0 on
            bits = n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u);
        } else {
            const uint64_t* m = a.mask + static_cast<size_t>(s.row0 + i) * a.mask_words;
            if (j0 < 0) {
                bits = static_cast<uint32_t>(m[0] << -j0) | ((1u << -j0) - 1u);
            } else {
                const int w = j0 >> 6, o = j0 & 63;
                uint64_t v = w < a.mask_words ? m[w] >> o : 0;
                if (o > 32 && w + 1 < a.mask_words) v |= m[w + 1] << (64 - o);
                bits = static_cast<uint32_t>(v);
            }
        }
    }
    const int left = end - c0;
    if (left < 32) bits &= left <= 0 ? 0u : (1u << left) - 1u;
    return bits;
}

// What is left to join of an item that begins in a block's share and ends in a later one.
struct JoinItem {
    int parts;                           // shares that hold a part of it; 0: nothing to join
    int row0, rows;                      // of the sequence: first row, packed rows of a kv head
    int h, mt;
};

// Partial results of a share: slot 2 * block + 1 for an item that begins in the block's
// share, 2 * block for one that began before it.
struct Partials {
    JoinItem* items;                     // [blocks]
    float* ml;                           // [slots][M][2]: maximum (base 2), sum
    float* o;                            // [slots][M][head_dim]
};

// shares from the one numbered `share` up to the one that holds the last of steps [.., end)
__device__ __forceinline__ int parts_until(long long W, int shares, int share, long long end) {
    return static_cast<int>((shares * end + W - 1) / W) - share;
}

constexpr int kSmallBlocks = 320;        // most blocks of the 16- to 64-row kernel
constexpr int kSmallRows = 64;
constexpr int kTileBlocks = 160;         // most blocks of the 256-row kernel
constexpr int kTileRows = 256;

cudaError_t launch_tree_attn_small(const AttnArgs& a, void* partials, cudaStream_t st);
cudaError_t launch_tree_attn_join(const AttnArgs& a, int M, Partials p, int blocks, cudaStream_t st);
// where the partial results of up to `blocks` blocks with tiles of M rows lie in memory
Partials partials_at(void* mem, int blocks, int M);
size_t partials_bytes(int blocks, int M, int head_dim);
bool make_kv_map(CUtensorMap* m, const AttnArgs& a, bool v, int box_rows, bool all_spans);
bool tree_attn_tiles_apply(const AttnArgs& a);
cudaError_t launch_tree_attn_tiles(const AttnArgs& a, void* partials, cudaStream_t st);

}  // namespace sre
