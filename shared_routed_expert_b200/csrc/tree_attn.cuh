// Attention over a paged cache: what its kernels share.
#pragma once

#include <cuda.h>

#include "kv_cache.cuh"

namespace sre {

struct AttnArgs {
    KvView c;
    int T, n_q, group;                   // group: query heads per kv head
    uint32_t group_mul, group_shift;     // r / group = mulhi(r, group_mul) >> group_shift for 0 <= r < 2^31
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

__device__ __forceinline__ int token_of(const AttnArgs& a, int r) {
    return a.group == 1 ? r : static_cast<int>(__umulhi(static_cast<uint32_t>(r), a.group_mul) >> a.group_shift);
}

// new rows that a sequence may have (rows behind the mask's columns are refused)
__device__ __forceinline__ int attn_max_new(const AttnArgs& a) {
    return a.mask != nullptr ? min(a.c.max_new, 64 * a.mask_words) : a.c.max_new;
}

// whether new token i of a sequence (row t of the call) sees the sequence's new token j
__device__ __forceinline__ bool sees_new(const AttnArgs& a, int t, int i, int j) {
    if (a.mask == nullptr) return j <= i;
    return (a.mask[static_cast<size_t>(t) * a.mask_words + (j >> 6)] >> (j & 63)) & 1;
}

// (special-function unit: 2 ulp; what goes through it is rounded to bf16, or a sum whose logarithm is taken)
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2F = 0.6931471805599453f;

// Exponents of P over E4M3 caches are raised by this much (of l and O with them), since P is fp16 there: the
// running maximum may lie 2^8 below the row's, so P stays below 2^15, and the smallest step of a weight is
// 2^-31 of the largest, not 2^-24 (a million keys of 2^-25 each would vanish from O, though not from l).
// bf16 has the exponents of fp32.
constexpr float kLift = 7.f;
template <bool F8>
__device__ __forceinline__ float lifted(float ref) {               // what a score's exponent is taken from
    if constexpr (F8) return ref - kLift;
    else return ref;
}

// ln sum 2^s from the maximum m (base 2) and l = sum 2^(s - m); -infinity for l = 0
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : (m + __log2f(l)) * kLn2F; }

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

// Whether one of the keys [lo, hi) that a row (token i of the sequence; -1: one that sees no new token) does
// not see has a value with an infinity or NaN, a lane per key. If none has, a NaN in the row's result is its
// own, and there is nothing to compute again (one NaN among 4000 cached values, seen by all rows, made calls 4
// to 180 times as long).
template <int D, bool F8>
__device__ __forceinline__ bool hides_infinities(const AttnArgs& a, int b, const SeqInfo& s, int i, int kv_head, int lo, int hi,
                                              int lane) {
    // (a row sees every cached token, in a chain the new ones up to itself too)
    for (int c0 = max(lo, a.mask != nullptr ? s.ctx : s.ctx + i + 1); c0 < hi; c0 += 32) {
        const int c = c0 + lane;
        bool found = false;
        if (c < hi && (i < 0 || !sees_new(a, s.row0 + i, i, c - s.ctx))) {
            const long long off = slot_offset(a.c, b, c, kv_head);
            for (int j = 0; off >= 0 && j < D * (F8 ? 1 : 2) / 16 && !found; ++j) {
                const uint4 v = *reinterpret_cast<const uint4*>(a.c.v + off + 16 * j);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if constexpr (F8) found |= __vcmpeq4(w[e] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
                    else found |= (w[e] & 0x7F80u) == 0x7F80u || (w[e] & 0x7F800000u) == 0x7F800000u;
                }
            }
        }
        if (__any_sync(0xFFFFFFFFu, found)) return true;
    }
    return false;
}

// ---- splitting the work
// An item is (sequence, kv head, tile of M query rows); the rows of a kv head are
// packed token-major, row r being token r / group, query head r % group. An item takes
// steps of SK keys up to the last key that one of its rows may see, and as much time as
// `extra` steps more for its beginning and end. These units of all items, in the order
// sequence, head, tile, are one axis that is cut into equal shares, one per block, so the
// load is even whatever the lengths; an item that a cut goes through leaves partial results
// (unnormalised sums with their maximum) that are joined in the order of the keys.

struct Tiling {
    int M, SK, extra;
};

// last cache index + 1 that rows of tile mt may see
__device__ __forceinline__ int tile_keys(const AttnArgs& a, const SeqInfo& s, int mt, int M) {
    if (a.mask != nullptr) return s.ctx + s.n;
    const int last = min((mt + 1) * M, s.n * a.group) - 1;
    return s.ctx + token_of(a, last) + 1;
}
__device__ __forceinline__ int tile_steps(const AttnArgs& a, const SeqInfo& s, int mt, Tiling g) {
    return (tile_keys(a, s, mt, g.M) + g.SK - 1) / g.SK;
}
__device__ __forceinline__ int seq_tiles(const AttnArgs& a, const SeqInfo& s, int M) {
    return (s.n * a.group + M - 1) / M;
}
// units of one kv head of a sequence
__device__ __forceinline__ long long head_units(const AttnArgs& a, const SeqInfo& s, Tiling g) {
    const int tiles = seq_tiles(a, s, g.M);
    if (tiles == 0) return 0;
    const int lo = tile_steps(a, s, 0, g), hi = tile_steps(a, s, tiles - 1, g);
    if (lo == hi) return static_cast<long long>(tiles) * (lo + g.extra);
    long long sum = 0;
    for (int mt = 0; mt < tiles; ++mt) sum += tile_steps(a, s, mt, g) + g.extra;
    return sum;
}

__device__ __forceinline__ long long div_pos(long long a, long long b) {       // a >= 0, b > 0
    return ((a | b) >> 31) ? a / b : static_cast<long long>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// W units cut into `count` shares, the first `longer` of them a unit longer.
struct Shares {
    int count, longer;
    long long base;

    __device__ __forceinline__ Shares(long long W, int blocks, int least) {
        const long long most = div_pos(W + least - 1, least);
        count = static_cast<int>(most < blocks ? most : blocks);
        base = count > 0 ? div_pos(W, count) : 0;
        longer = static_cast<int>(W - base * count);
    }
    __device__ __forceinline__ long long begin(int i) const { return i * base + min(i, longer); }
    __device__ __forceinline__ int of(long long x) const {                     // the share that holds unit x
        const long long head = longer * (base + 1);
        return static_cast<int>(x < head ? div_pos(x, base + 1) : longer + div_pos(x - head, base));
    }
};

struct ScanShared {
    long long warp_sum[32];
    long long rem, per;                  // of the sequence that was looked for: units in front, units of a head
    SeqInfo s;
    int b;
};

// A thread's part of the scan: its sequences [b0, b1), the units in front of them, and the
// first one's lengths
struct ScanThread {
    long long before, per;
    int b0, b1;
    SeqInfo s;
};

// All units of the call; called by every thread of the block.
__device__ __forceinline__ long long scan_units(const AttnArgs& a, Tiling g, ScanShared& sh, ScanThread& me) {
    const int each = (a.c.B + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    me.b0 = min(a.c.B, static_cast<int>(threadIdx.x) * each);
    me.b1 = min(a.c.B, me.b0 + each);
    long long mine = 0;
    for (int b = me.b0; b < me.b1; ++b) {
        const SeqInfo s = seq_info(a.c, b, a.T, attn_max_new(a));
        if (!s.ok && blockIdx.x == 0) report(a.status, MOE_ERR_DEVICE, b);
        const long long per = head_units(a, s, g);
        if (b == me.b0) {
            me.s = s;
            me.per = per;
        }
        mine += per * a.c.n_kv;
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
    me.before = base + inc - mine;
    return W;
}

// A place on the axis: an item and the unit within it.
struct Cursor {
    SeqInfo s;
    int b, h, mt, unit, steps;           // steps: of the whole item

    // to the first unit of the next item (sequences without rows are passed over)
    __device__ __forceinline__ void next(const AttnArgs& a, Tiling g) {
        unit = 0;
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
        steps = tile_steps(a, s, mt, g);
    }
    // Moves on to the next item with steps inside the share (`left` units from here): its
    // steps [lo, hi); false at the end of the share. The cursor then stands behind hi.
    __device__ __forceinline__ bool segment(const AttnArgs& a, Tiling g, long long& left, int& lo, int& hi) {
        while (left > 0) {
            if (unit >= g.extra + steps) next(a, g);
            const int to = static_cast<int>(min(static_cast<long long>(g.extra + steps), unit + left));
            lo = max(0, unit - g.extra);
            hi = max(0, to - g.extra);
            left -= to - unit;
            unit = to;
            if (hi > lo) return true;
        }
        return false;
    }
};

// The place of unit x (0 <= x < W), by every thread of the block, after scan_units.
__device__ __forceinline__ Cursor seek(const AttnArgs& a, Tiling g, ScanShared& sh, long long x, const ScanThread& me) {
    if (x >= me.before) {
        long long rem = x - me.before;
        SeqInfo s = me.s;
        long long per = me.per;
        for (int b = me.b0; b < me.b1; ++b) {
            if (b > me.b0) {
                s = seq_info(a.c, b, a.T, attn_max_new(a));
                per = head_units(a, s, g);
            }
            if (rem < per * a.c.n_kv) {
                sh.b = b;
                sh.s = s;
                sh.rem = rem;
                sh.per = per;
                break;
            }
            rem -= per * a.c.n_kv;
        }
    }
    __syncthreads();
    Cursor c;
    c.b = sh.b;
    c.s = sh.s;
    const long long per = sh.per;
    c.h = static_cast<int>(div_pos(sh.rem, per));
    long long rem = sh.rem - c.h * per;
    c.mt = 0;
    c.steps = tile_steps(a, c.s, 0, g);
    const int units = c.steps + g.extra;
    if (per == static_cast<long long>(units) * seq_tiles(a, c.s, g.M)) {
        c.mt = static_cast<int>(div_pos(rem, units));
        rem -= static_cast<long long>(c.mt) * units;
    } else {
        while (rem >= c.steps + g.extra) {
            rem -= c.steps + g.extra;
            ++c.mt;
            c.steps = tile_steps(a, c.s, c.mt, g);
        }
    }
    c.unit = static_cast<int>(rem);
    return c;
}

// The shares that hold steps of the item that a cursor behind some of its units stands in
// (`end`: the share's end, `left`: what is left of it): the first one and their number.
__device__ __forceinline__ int2 item_shares(const Shares& sh, const Cursor& c, Tiling g, long long end, long long left) {
    const long long start = end - left - c.unit + g.extra;
    const int first = sh.of(start);
    return make_int2(first, sh.of(start + c.steps - 1) - first + 1);
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
    unsigned* arrived;                   // [blocks] parts of the item that begins in a share; 0 between calls
    JoinItem* items;                     // [blocks]
    float* ml;                           // [slots][M][2]: maximum (base 2), sum
    float* o;                            // [slots][M][head_dim]
};

// Row r of a tile of M rows (rr of the item's packed rows) from its parts in `parts` shares
// from `first` on, by one warp: with m = max m_p, sum_p 2^{m_p - m} (l_p, o_p); the loads of
// AT_ONCE parts are in flight together.
template <int EPL, int AT_ONCE>
__device__ __forceinline__ void join_row(const AttnArgs& a, const Partials& p, int M, int first, int parts, int row0, int h,
                                         int r, int rr, int lane) {
    auto slot = [&](int i) { return 2 * static_cast<size_t>(first + i) + (i == 0); };
    float m = -INFINITY;
    float2 own = make_float2(-INFINITY, 0.f);                      // lane i: part i's (of the first 32)
    for (int i = lane; i < parts; i += 32) {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(p.ml + (slot(i) * M + r) * 2));
        if (i < 32) own = v;
        m = fmaxf(m, v.x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, acc[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) acc[j] = 0.f;
    for (int p0 = 0; p0 < parts; p0 += 32) {
        if (p0 > 0) own = p0 + lane < parts ? __ldcg(reinterpret_cast<const float2*>(p.ml + (slot(p0 + lane) * M + r) * 2)) : make_float2(-INFINITY, 0.f);
        const float f = fast_exp2(own.x - ref);
        l += own.y * f;
        const int n = min(32, parts - p0);
        // (behind the last part the weights are 0)
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += AT_ONCE) {
#pragma unroll
            for (int e = 0; e < AT_ONCE; ++e) {
                const size_t at = slot(p0 + min(i0 + e, n - 1)) * M + r;
                const float w = __shfl_sync(0xFFFFFFFFu, f, i0 + e);
                float o[EPL];
                if constexpr (EPL == 2) {
                    *reinterpret_cast<float2*>(o) = __ldcg(reinterpret_cast<const float2*>(p.o + at * 64) + lane);
                } else {
#pragma unroll
                    for (int q = 0; q < EPL / 4; ++q)
                        *reinterpret_cast<float4*>(o + 4 * q) =
                            __ldcg(reinterpret_cast<const float4*>(p.o + at * (32 * EPL)) + lane * (EPL / 4) + q);
                }
                if (i0 + e < n) {
#pragma unroll
                    for (int j = 0; j < EPL; ++j) acc[j] += o[j] * w;
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
    const int i = token_of(a, rr), head = h * a.group + rr - i * a.group;
    const long long row = row0 + i;
    const float inv = l == 0.f ? 0.f : __fdividef(a.c.v_scale, l);
    uint32_t w[EPL / 2];
#pragma unroll
    for (int j = 0; j < EPL; j += 2) w[j / 2] = l == 0.f ? 0u : pack_bf16x2(acc[j] * inv, acc[j + 1] * inv);
    uint16_t* dst = a.out + row * a.out_stride + head * (32 * EPL) + lane * EPL;
    if constexpr (EPL == 2) *reinterpret_cast<uint32_t*>(dst) = w[0];
    else if constexpr (EPL == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[EPL / 2 - 2], w[EPL / 2 - 1]);
    if (a.lse != nullptr && lane == 0) a.lse[row * a.n_q + head] = lse_of(m, l);
}

// pairs of fp32 in one register pair: one instruction for two multiply-adds or additions
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// Of the lanes `lanes`, those whose row's NaN may come from a value that it does not see (the lanes hold rows
// of the item in order, i their tokens).
template <int D, bool F8>
__device__ __noinline__ uint32_t spoiled_lanes(const AttnArgs& a, const Cursor& c, int i, uint32_t lanes, int lo, int hi, int lane) {
    // first for a row that sees no more than any of them: mostly there is no such value
    const int first = __shfl_sync(0xFFFFFFFFu, i, __ffs(lanes) - 1);
    if (!hides_infinities<D, F8>(a, c.b, c.s, a.mask != nullptr ? -1 : first, c.h, lo, hi, lane)) return 0;
    uint32_t yes = 0;
#pragma unroll 1
    for (uint32_t rest = lanes; rest; rest &= rest - 1) {
        const int src = __ffs(rest) - 1;
        if (hides_infinities<D, F8>(a, c.b, c.s, __shfl_sync(0xFFFFFFFFu, i, src), c.h, lo, hi, lane)) yes |= 1u << src;
    }
    return yes;
}
// A row of an item again, key by key (a rare path, kept out of the main code's registers)
template <int D, bool F8>
__device__ __forceinline__ void redo_row(const AttnArgs& a, const Cursor& c, int i, int head, int lo, int hi, float* o, float* ml,
                                      int lane) {
    constexpr int EPL = D / 32;
    float q[EPL], acc[EPL], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
        q[j] = bf16_to_f32(a.q[(c.s.row0 + i) * a.q_stride + head * D + lane * EPL + j]);
        acc[j] = 0.f;
    }
    attend_row<EPL, F8>(a, c.b, c.s, i, c.h, q, lo, hi, m, l, acc, lane);
    if (o != nullptr) {
#pragma unroll
        for (int j = 0; j < EPL; ++j) o[lane * EPL + j] = acc[j];
        if (lane == 0) {
            ml[0] = m;
            ml[1] = l;
        }
    } else {
        const long long row = c.s.row0 + i;
        const float inv = l == 0.f ? 0.f : __fdividef(a.c.v_scale, l);
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            a.out[row * a.out_stride + head * D + lane * EPL + j] = f32_to_bf16(l == 0.f ? 0.f : acc[j] * inv);
        if (a.lse != nullptr && lane == 0) a.lse[row * a.n_q + head] = lse_of(m, l);
    }
}

// The rows of the lanes `lanes` that spoiled_lanes names, again: into out, or (part_o and part_ml not null)
// into the partial results from this warp's first row on
template <int D, bool F8>
__device__ __noinline__ void redo_rows(const AttnArgs& a, const Cursor& c, uint32_t lanes, int i, int head, int lo, int hi,
                                       float* part_o, float* part_ml, int lane) {
#pragma unroll 1
    for (uint32_t rest = spoiled_lanes<D, F8>(a, c, i, lanes, lo, hi, lane); rest; rest &= rest - 1) {
        const int src = __ffs(rest) - 1;
        redo_row<D, F8>(a, c, __shfl_sync(0xFFFFFFFFu, i, src), __shfl_sync(0xFFFFFFFFu, head, src), lo, hi,
                        part_o == nullptr ? nullptr : part_o + src * D, part_ml + src * 2, lane);
    }
}

constexpr int kSmallBlocks = 320;        // most blocks of the 16- or 32-row kernel
constexpr int kSmallRows = 32;
constexpr int kTileBlocks = 160;         // most blocks of the 256- and 128-row kernels
constexpr int kTileRows = 256;
constexpr int kWideRows = 128;           // ... of heads of 256 dimensions

cudaError_t launch_tree_attn_small(const AttnArgs& a, void* partials, cudaStream_t st);
cudaError_t launch_tree_attn_join(const AttnArgs& a, int M, Partials p, int blocks, cudaStream_t st);
// where the partial results of up to `blocks` blocks with tiles of M rows lie in memory
Partials partials_at(void* mem, int blocks, int M);
size_t partials_bytes(int blocks, int M, int head_dim);
// Cycles after which a wait of the tile kernels gives up: 9 s, and what a warp may spend on computing 32 rows
// again behind as many keys as the page table holds (8192 cycles a row and key; 1200 were measured where they
// come from L2, heads of 256), while the others wait for it
long long tile_wait_limit(const AttnArgs& a);
bool make_kv_map(CUtensorMap* m, const AttnArgs& a, bool v, int box_rows);
// testing hook: the next n calls run with loads that are never issued and a ~10 ms wait limit
void tree_attn_inject_stall(int n_calls);
bool tree_attn_take_stall();
// whether a call is so short that the 16- or 32-row kernel takes it whatever its rows
bool tree_attn_short(const AttnArgs& a);
bool tree_attn_tiles_apply(const AttnArgs& a);
bool tree_attn_wide_apply(const AttnArgs& a);
cudaError_t launch_tree_attn_tiles(const AttnArgs& a, void* partials, cudaStream_t st);
cudaError_t launch_tree_attn_wide(const AttnArgs& a, void* partials, cudaStream_t st);

}  // namespace sre
