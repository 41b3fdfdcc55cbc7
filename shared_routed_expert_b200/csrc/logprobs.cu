// Log probabilities of given tokens, entropy and the likeliest alternatives of rows
// of logits, in one pass over the logits.
//
// With M the row's largest logit, one occurrence of it left out of the sums,
//   l = sum e^{x-M},  t = sum e^{x-M} (M - x)       (over the other V - 1 terms)
//   ln sum e^x = M + ln(1 + l),  entropy = ln(1 + l) + t / (1 + l),
// so a row with one likely token keeps the relative accuracy of l. The pass works
// in base 2 (d = (x - m) log2 e with the running maximum m of the thread).
//
// A row is read by a cluster of C blocks, each a slice of it; a thread reads groups
// of kU 16-byte vectors and keeps, besides the running sums, the largest value of
// each of its (at most kG) runs of groups in shared memory. The sums of the group
// that brought the maximum stay apart from the rest, so that leaving out one
// occurrence of the maximum costs one more read of one group at the end.
//
// Alternatives: the n-th largest of the threads' maxima bounds the n-th largest
// element from below, so only runs whose maximum reaches it are read again (about
// n of them, from L2), and the elements that reach it are ranked by (value
// descending, id ascending). Rows where more elements than the list holds reach
// the bound, or that hold NaN or +infinity, take n rounds over the slice instead. Rows with fewer
// threads that hold an unmasked logit than alternatives are among them: 131072 bf16 logits, 20
// alternatives, 62 us with 1 to 10 tokens left and 11 us with 1000 (or none masked).
//
// Bound by HBM for many rows (each logit is read once): 2048 rows of 100003 fp32, 819 MB, 158 us,
// 5.2 TB/s (166 us back to back; blocks of 512 threads: 187 us; smaller ones hide each other's ends of rows). By
// latency for a few: one row of 131072 bf16 with 20 alternatives 9.8 us. bf16 rows are bound by
// the instructions per logit: 2048 rows of 100003 115 us, 3.6 TB/s.
#include <cooperative_groups.h>

#include "kernels.cuh"

namespace sre {

namespace {

namespace cg = cooperative_groups;

constexpr int LP_THREADS = 256;
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int kU = 4;                    // 16-byte vectors per group
constexpr int kG = 16;                   // runs of groups per thread
constexpr int kTop = 32;                 // most alternatives
constexpr int kCand = 512;               // candidates a block ranks
constexpr int kMaxC = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
static_assert(kMaxC <= LP_WARPS && kTop == 32, "the join has a warp per slice and a lane per alternative");

// order-preserving key: larger values have larger keys, NaN the largest, -0 = +0
__device__ __forceinline__ uint32_t value_key(float x) {
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(x + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}
// (value, id) as one number: larger = ranked first
__device__ __forceinline__ unsigned long long pair_key(float x, int id) {
    return (static_cast<unsigned long long>(value_key(x)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(id));
}
__device__ __forceinline__ int pair_id(unsigned long long k) {
    return static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(k));
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// From reference `from` down to a larger one, base 2. Bounded: a sum times it stays finite where its power is
// 0 (a mask of the type's lowest value overflows it to -infinity, and -infinity * 0 is NaN).
__device__ __forceinline__ float fall(float from, float to) { return fmaxf((from - to) * kLog2e, -1000.0f); }

// pairs of fp32 in one register pair
__device__ __forceinline__ uint64_t pair2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// a thread's sums against its reference (its maximum, or 0 while everything is -infinity)
struct Sums {
    float l, t;                          // sum e, sum e * d (base 2, d <= 0)
};

template <bool BF16>
struct Row {
    static constexpr int VE = BF16 ? 8 : 4;                        // elements per vector
    static constexpr int GE = VE * kU;                             // elements per group
    const char* p;                       // the row
    int V;
    int head;                            // elements in front of the first 16-byte boundary

    __device__ __forceinline__ float at(int i) const {
        if constexpr (BF16) return bf16_to_f32(reinterpret_cast<const uint16_t*>(p)[i]);
        else return reinterpret_cast<const float*>(p)[i];
    }
    __device__ __forceinline__ uint4 vec(int v) const {            // vector v behind the head
        return __ldg(reinterpret_cast<const uint4*>(p + static_cast<size_t>(head) * (BF16 ? 2 : 4)) + v);
    }
    static __device__ __forceinline__ void widen(const uint4& w, float* f) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (BF16) {
                f[2 * j] = __uint_as_float(u[j] << 16);
                f[2 * j + 1] = __uint_as_float(u[j] & 0xFFFF0000u);
            } else {
                f[j] = __uint_as_float(u[j]);
            }
        }
    }
};

struct LpShared {
    float run_max[kG][LP_THREADS];
    unsigned long long cand[kCand];
    unsigned long long top[kTop];        // this block's alternatives, best first
    unsigned long long warp_top[LP_WARPS][32];
    uint32_t warp_key[LP_WARPS][32];
    float red[LP_WARPS][4];
    float4 part[kMaxC];                  // rank 0: the slices' m, l, t, bad
    float4 sums;                         // this block's maximum, its sums without one maximum, and whether
                                         // the slice holds NaN or +infinity
    int n_cand;
};

// Sorted lists of 32 over a warp's lanes, largest first.
template <typename K>
__device__ __forceinline__ K sort_desc_warp(K k, int lane) {
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
        for (int j = size >> 1; j > 0; j >>= 1) {
            const K o = __shfl_xor_sync(0xFFFFFFFFu, k, j);
            const bool first = (lane & j) == 0, desc = (lane & size) == 0 || size == 32;
            k = (first == desc) ? (k > o ? k : o) : (k < o ? k : o);
        }
    }
    return k;
}
// a, b sorted -> the 32 largest of both, sorted
template <typename K>
__device__ __forceinline__ K merge_desc_warp(K a, K b, int lane) {
    const K r = __shfl_sync(0xFFFFFFFFu, b, 31 - lane);
    K k = a > r ? a : r;                                           // bitonic, holds the 32 largest
#pragma unroll
    for (int j = 16; j > 0; j >>= 1) {
        const K o = __shfl_xor_sync(0xFFFFFFFFu, k, j);
        k = ((lane & j) == 0) ? (k > o ? k : o) : (k < o ? k : o);
    }
    return k;
}
// the 32 largest of the block's sorted lists (one per warp), to lists[0]
template <typename K>
__device__ __forceinline__ void merge_block(K (*lists)[32], K k, int warp, int lane) {
    lists[warp][lane] = k;
    __syncthreads();
#pragma unroll
    for (int w = LP_WARPS / 2; w > 0; w >>= 1) {
        if (warp < w) lists[warp][lane] = merge_desc_warp(lists[warp][lane], lists[warp + w][lane], lane);
        __syncthreads();
    }
}

__device__ __forceinline__ unsigned long long block_max(LpShared& sh, unsigned long long k, int warp, int lane) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long x = __shfl_xor_sync(0xFFFFFFFFu, k, o);
        k = x > k ? x : k;
    }
    __syncthreads();
    if (lane == 0) sh.warp_top[0][warp] = k;
    __syncthreads();
    unsigned long long b = 0;
#pragma unroll
    for (int w = 0; w < LP_WARPS; ++w) b = sh.warp_top[0][w] > b ? sh.warp_top[0][w] : b;
    return b;
}

template <bool BF16>
__global__ void __launch_bounds__(LP_THREADS, 4) logprobs_kernel(int V, const char* __restrict__ logits,
                                                              long long row_b, const int32_t* __restrict__ targets,
                                                              int top_n, float* __restrict__ logprobs,
                                                              float* __restrict__ entropy, int32_t* __restrict__ top_ids,
                                                              float* __restrict__ top_lp) {
    using R = Row<BF16>;
    constexpr int ESZ = BF16 ? 2 : 4;
    __shared__ LpShared sh;
    const cg::cluster_group cl = cg::this_cluster();
    const int C = cl.num_blocks(), rank = cl.block_rank();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int t = blockIdx.x / C;

    R row;
    row.p = logits + t * row_b;
    row.V = V;
    row.head = min(V, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(row.p) & 15)) & 15) / ESZ);
    const int n_vec = (V - row.head) / R::VE;
    // this block's vectors, and the scalars in front of and behind them
    const int v_lo = static_cast<int>(static_cast<long long>(n_vec) * rank / C);
    const int v_hi = static_cast<int>(static_cast<long long>(n_vec) * (rank + 1) / C);
    const int tail0 = row.head + n_vec * R::VE;
    const int groups = (v_hi - v_lo + kU * LP_THREADS - 1) / (kU * LP_THREADS);   // groups per thread
    const int per_run = max(1, (groups + kG - 1) / kG);
    if (tid == 0) {
        sh.n_cand = 0;
    }

    // ---- one pass: m, rest (without the best group), best
    float m = -INFINITY;
    Sums rest{0.f, 0.f}, best{0.f, 0.f};
    int best_g = -1;                     // group of the maximum; -2: the thread's scalar
    float run = -INFINITY;
    auto account = [&](const auto& f, float gm, int g) {
        constexpr int n = sizeof(f) / sizeof(float);
        // sums of the group against the reference after it
        const float m2 = fmaxf(m, gm);
        const float ref = m2 == -INFINITY ? 0.0f : m2;
        if (gm > m) {
            const float shift = m == -INFINITY ? 0.0f : fall(m, ref);   // <= 0
            const float a = exp2_fast(shift);
            const float l = rest.l + best.l;
            rest.t = (rest.t + best.t + l * shift) * a;
            rest.l = l * a;
        }
        float l = 0.f, tt = 0.f;
        if constexpr (n % 4 == 0) {
            // pairs, one instruction each; the difference first: exact near the maximum
            const uint64_t r2 = pair2(-ref, -ref), c2 = pair2(kLog2e, kLog2e);
            uint64_t l2[2] = {0, 0}, t2[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < n; j += 2) {
                const uint64_t d2 = mul2(add2(pair2(f[j], f[j + 1]), r2), c2);
                float da, db;
                unpair2(d2, da, db);
                const uint64_t e2 = pair2(exp2_fast(da), exp2_fast(db));
                l2[(j >> 1) & 1] = add2(l2[(j >> 1) & 1], e2);
                t2[(j >> 1) & 1] = fma2(e2, d2, t2[(j >> 1) & 1]);
            }
            float x, y;
            unpair2(add2(l2[0], l2[1]), x, y);
            l = x + y;
            unpair2(add2(t2[0], t2[1]), x, y);
            tt = x + y;
        }
        if (n % 4 != 0 || tt != tt) {
            // one by one, with -infinity (where 0 * d is not 0) looked after
            l = tt = 0.f;
#pragma unroll
            for (int j = 0; j < n; ++j) {
                const float d = (f[j] - ref) * kLog2e;
                const float e = exp2_fast(d);
                l += e;
                tt = fmaf(e, fmaxf(d, -1.0e30f), tt);
            }
        }
        if (gm > m) {
            best.l = l;
            best.t = tt;
            best_g = g;
            m = gm;
        } else {
            rest.l += l;
            rest.t += tt;
        }
    };
    // scalars: thread s < head takes element s (rank 0), threads behind it the tail (last rank)
    int scalar = -1;
    if (rank == 0 && tid < row.head) scalar = tid;
    const int n_tail = V - tail0;
    if (rank == C - 1 && tid >= 32 && tid - 32 < n_tail) scalar = tail0 + tid - 32;
    if (scalar >= 0) {
        const float f[1] = {row.at(scalar)};
        account(f, f[0], -2);
        run = m;
    }
    int run_i = 0;
    uint4 w[kU];
    auto fetch = [&](int g) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int v = v_lo + g * (kU * LP_THREADS) + tid + u * LP_THREADS;
            if (g < groups && v < v_hi) w[u] = row.vec(v);
            else w[u] = BF16 ? make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u)
                             : make_uint4(0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u);   // -infinity
        }
    };
    fetch(0);
    int target = -1;
    float x_target = 0.f;
    if (rank == 0 && tid == 0 && logprobs != nullptr) {
        target = targets[t];
        if (target >= 0 && target < V) x_target = row.at(target);
    }
    for (int g = 0; g < groups; ++g) {
        float f[R::GE];
#pragma unroll
        for (int u = 0; u < kU; ++u) R::widen(w[u], f + u * R::VE);
        fetch(g + 1);                                              // on its way while this group is summed
        float gm = f[0], gm2 = f[1];
#pragma unroll
        for (int j = 2; j < R::GE; j += 4) {
            gm = fmaxf(fmaxf(gm, f[j]), f[j + 1]);
            if (j + 2 < R::GE) gm2 = fmaxf(fmaxf(gm2, f[j + 2]), f[j + 3]);
        }
        gm = fmaxf(gm, gm2);
        account(f, gm, g);
        run = fmaxf(run, gm);
        if ((g + 1) % per_run == 0 || g + 1 == groups) {
            sh.run_max[run_i++][tid] = run;
            run = -INFINITY;
        }
    }
    if (groups == 0) {
        sh.run_max[0][tid] = run;
        run_i = 1;
    }

    // ---- the block's maximum and sums
    float bm = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xFFFFFFFFu, bm, o));
    if (lane == 0) sh.red[warp][0] = bm;
    __syncthreads();
    bm = sh.red[0][0];
#pragma unroll
    for (int w = 1; w < LP_WARPS; ++w) bm = fmaxf(bm, sh.red[w][0]);
    // the lowest thread that holds the maximum leaves one occurrence out
    const unsigned has = __ballot_sync(0xFFFFFFFFu, m == bm && best_g != -1);
    if (lane == 0) sh.red[warp][1] = __uint_as_float(has);
    __syncthreads();
    int owner = -1;
#pragma unroll
    for (int w = LP_WARPS - 1; w >= 0; --w) {
        const unsigned hw = __float_as_uint(sh.red[w][1]);
        if (hw) owner = w * 32 + __ffs(hw) - 1;
    }
    const float bref = bm == -INFINITY ? 0.0f : bm;
    uint4 again[kU];                                               // the owner's best group, on its way while the alternatives are found
    if (tid == owner && best_g >= 0) {
#pragma unroll
        for (int u = 0; u < kU; ++u) {
            const int v = v_lo + best_g * (kU * LP_THREADS) + tid + u * LP_THREADS;
            again[u] = v < v_hi ? row.vec(v) : make_uint4(0, 0, 0, 0);
        }
    }

    // ---- this block's alternatives (rows with NaN or +infinity: see below)
    const bool odd = __syncthreads_or(!(rest.l + best.l < INFINITY)) || bm == INFINITY;
    if (top_n > 0) {
        bool rounds = odd;
        if (!rounds) {
            // the n-th largest of the threads' maxima
            float tau = bm;
            if (top_n > 1) {
                merge_block(sh.warp_key, sort_desc_warp(value_key(m), lane), warp, lane);
                tau = key_value(sh.warp_key[0][top_n - 1]);
            }
            auto offer = [&](float x, int id) {
                const int i = atomicAdd(&sh.n_cand, 1);
                if (i < kCand) sh.cand[i] = pair_key(x, id);
            };
            if (m >= tau) {
                if (scalar >= 0) {
                    const float x = row.at(scalar);
                    if (x >= tau) offer(x, scalar);
                }
                for (int r = 0; r < run_i; ++r) {
                    if (groups == 0 || !(sh.run_max[r][tid] >= tau)) continue;
                    for (int g = r * per_run; g < min(groups, (r + 1) * per_run); ++g) {
                        uint4 q[kU];
#pragma unroll
                        for (int u = 0; u < kU; ++u) {
                            const int v = v_lo + g * (kU * LP_THREADS) + tid + u * LP_THREADS;
                            if (v < v_hi) q[u] = row.vec(v);
                        }
#pragma unroll
                        for (int u = 0; u < kU; ++u) {
                            const int v = v_lo + g * (kU * LP_THREADS) + tid + u * LP_THREADS;
                            float f[R::VE];
                            R::widen(q[u], f);
                            unsigned hit = 0;
#pragma unroll
                            for (int j = 0; j < R::VE; ++j) hit |= (f[j] >= tau ? 1u : 0u) << j;
                            if (v >= v_hi) hit = 0;
                            while (hit) {
                                const int j = __ffs(hit) - 1;
                                hit &= hit - 1;
                                const int id = row.head + v * R::VE + j;
                                offer(row.at(id), id);
                            }
                        }
                    }
                }
            }
            __syncthreads();
            const int n = sh.n_cand;
            rounds = n > kCand;
            if (!rounds) {
                if (tid < kTop) sh.top[tid] = 0;
                __syncthreads();
                for (int i = tid; i < n; i += LP_THREADS) {
                    const unsigned long long k = sh.cand[i];
                    int r = 0;
#pragma unroll 8
                    for (int j = 0; j < n; ++j) r += sh.cand[j] > k;
                    if (r < top_n) sh.top[r] = k;
                }
            }
        }
        if (rounds) {
            if (tid < kTop) sh.top[tid] = 0;
            unsigned long long last = ~0ull;
            for (int i = 0; i < top_n; ++i) {
                unsigned long long k = 0;
                auto look = [&](float x, int id) {
                    const unsigned long long p = pair_key(x, id);
                    if ((p < last || i == 0) && p > k) k = p;
                };
                if (scalar >= 0) look(row.at(scalar), scalar);
                for (int v = v_lo + tid; v < v_hi; v += LP_THREADS) {
                    float f[R::VE];
                    R::widen(row.vec(v), f);
#pragma unroll
                    for (int j = 0; j < R::VE; ++j) look(f[j], row.head + v * R::VE + j);
                }
                last = block_max(sh, k, warp, lane);
                if (tid == 0) sh.top[i] = last;
            }
        }
    }

    // ---- the block's sums, the owner's best group without the first occurrence of the maximum
    if (tid == owner) {
        best.l = best.t = 0.f;
        if (best_g >= 0) {
            bool out = false;
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                if (v_lo + best_g * (kU * LP_THREADS) + tid + u * LP_THREADS >= v_hi) continue;
                float f[R::VE];
                R::widen(again[u], f);
#pragma unroll
                for (int j = 0; j < R::VE; ++j) {
                    if (!out && f[j] == bm) {
                        out = true;
                        continue;
                    }
                    const float d = (f[j] - bref) * kLog2e;
                    const float e = exp2_fast(d);
                    best.l += e;
                    best.t = fmaf(e, fmaxf(d, -1.0e30f), best.t);
                }
            }
        }
    }
    float l = rest.l + best.l, tt = rest.t + best.t;
    {
        const float shift = m == -INFINITY ? 0.0f : fall(m, bref);
        const float a = exp2_fast(shift);
        tt = (tt + l * shift) * a;
        l *= a;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        tt += __shfl_xor_sync(0xFFFFFFFFu, tt, o);
    }
    __syncthreads();                                               // red[..][1] has been read
    if (lane == 0) {
        sh.red[warp][2] = l;
        sh.red[warp][3] = tt;
    }
    __syncthreads();
    if (tid == 0) {
        l = tt = 0.f;
#pragma unroll
        for (int w = 0; w < LP_WARPS; ++w) {
            l += sh.red[w][2];
            tt += sh.red[w][3];
        }
        sh.sums = make_float4(bm, l, tt, odd ? 1.f : 0.f);
    }
    __syncthreads();

    // ---- join the slices
    if (C > 1) cl.sync();
    else __syncthreads();
    if (rank == 0) {
        // the slices' sums and alternatives, each read once: slice w's list by warp w
        if (tid < C) sh.part[tid] = C > 1 ? cl.map_shared_rank(&sh, tid)->sums : sh.sums;
        unsigned long long k = 0;
        if (C > 1) {
            if (top_n > 0) {
                merge_block(sh.warp_top, warp < C ? cl.map_shared_rank(&sh, warp)->top[lane] : 0ull, warp, lane);
                if (warp == 0) k = sh.warp_top[0][lane];
            } else {
                __syncthreads();
            }
        } else {
            __syncthreads();
            if (top_n > 0 && warp == 0) k = sh.top[lane];
        }
        float M = -INFINITY;
        bool bad = false;
        for (int r = 0; r < C; ++r) {
            M = fmaxf(M, sh.part[r].x);
            bad |= sh.part[r].w != 0.f;
        }
        bad |= M == -INFINITY;
        float L = 0.f, TT = 0.f;
        bool out = false;
        for (int r = 0; r < C; ++r) {
            const float4 o = sh.part[r];
            if (o.x == -INFINITY) continue;
            float ol = o.y;
            if (o.x == M && !out) out = true;                      // the one maximum left out
            else ol += 1.0f;
            const float shift = fall(o.x, M), a = exp2_fast(shift);
            TT += (o.z + ol * shift) * a;
            L += ol * a;
        }
        const float ln1 = log1pf(L);
        if (tid == 0) {
            if (logprobs != nullptr)
                logprobs[t] = (bad || target < 0 || target >= V) ? NAN : (x_target - M) - ln1;
            if (entropy != nullptr) entropy[t] = bad ? NAN : ln1 - TT * kLn2 / (1.0f + L);
        }
        if (warp == 0 && lane < top_n && k != 0) {
            top_ids[static_cast<long long>(t) * top_n + lane] = pair_id(k);
            top_lp[static_cast<long long>(t) * top_n + lane] = bad ? NAN : (key_value(static_cast<uint32_t>(k >> 32)) - M) - ln1;
        }
    }
    if (C > 1) cl.sync();                                          // rank 0 has read the others' memory
}

}  // namespace

cudaError_t launch_logprobs(int T, int V, bool bf16, const void* logits, long long row_stride, const int32_t* targets,
                            int top_n, float* logprobs, float* entropy, int32_t* top_ids, float* top_lp,
                            cudaStream_t st) {
    ProfileScope ps("token_logprobs", st);
    // blocks per row: few rows are spread over more SMs, while that makes no more than 3 blocks per SM with
    // slices of 8192 elements (160 rows of 128000 fp32: 23 us with 2 blocks, 32 with 1; 300 rows: 43 and 41),
    // or 1 per SM with slices of 4096 (12 rows of 32000 bf16: 5.7 us with 4 blocks, 6.5 with 2; 129 rows
    // of 11217: 6.6 with 2, 5.6 with 1)
    int C = 1;
    auto fits = [&](int blocks, int slice) { return static_cast<long long>(T) * 2 * C <= blocks && V / (2 * C) >= slice; };
    while (C < kMaxC && (fits(444, 8192) || fits(148, 4096))) C *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(T) * C);
    cfg.blockDim = dim3(LP_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const char* p = static_cast<const char*>(logits);
    const long long row_b = row_stride * (bf16 ? 2 : 4);
    const cudaError_t e = bf16 ? cudaLaunchKernelEx(&cfg, logprobs_kernel<true>, V, p, row_b, targets, top_n, logprobs,
                                                    entropy, top_ids, top_lp)
                               : cudaLaunchKernelEx(&cfg, logprobs_kernel<false>, V, p, row_b, targets, top_n, logprobs,
                                                    entropy, top_ids, top_lp);
    note_launch();
    return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace sre
