// Attention over a paged cache for few query rows per kv head (decoding, short drafts):
// bound by reading the cache once.
//
// Flash decoding with warp-level matrix instructions: a block takes tiles of M = 16, 32
// or 64 packed query rows and runs along its share of the key axis (tree_attn.cuh). A
// producer warp streams chunks of 32 keys (K and V rows, one TMA box per page piece)
// through a ring in shared memory; 4 / WM groups of WM warps take the chunks in turn,
// each warp 16 rows, with its own running maximum and sum, so warps meet only at the end
// of an item. Scores and the output accumulate in fp32 registers (m16n8k16); P is rounded
// to 16 bits as the second product's operand.
//   bf16 cache: Q, K, P, V as bf16.
//   E4M3 cache: K and V codes convert to fp16 exactly; Q rows are scaled by a power of two
//   to fp16 (exact for everything within 2^-28 of the row's largest entry) and P is fp16.
//   K's dimensions are taken in the order that lets a thread read 8 consecutive codes,
//   and V's 16-bit transposed loads return pairs of neighbouring dimensions that a byte
//   permutation turns into pairs of keys.
// The accumulators are rescaled only when a row's maximum grows by more than 2^8 (P stays
// below 2^8, far from fp16's and bf16's limits).
#include "kernels.cuh"
#include "tc_ptx.cuh"
#include "tree_attn.cuh"

namespace sre {

namespace {

constexpr int CK = 32;                   // keys per chunk
constexpr int SM_THREADS = 160;          // 4 compute warps and the producer

template <int D, bool F8, int WM>
struct Small {
    static constexpr int ESZ = F8 ? 1 : 2;
    static constexpr int M = 16 * WM, WK = 4 / WM, SK = CK * WK;
    static constexpr int ROWB = D * ESZ < 128 ? D * ESZ : 128;     // bytes of a row within one swizzle span
    static constexpr int KBYTES = CK * D * ESZ;                    // K (or V) of a chunk
    static constexpr int STAGE = 2 * KBYTES;
    static constexpr int RING = D == 256 ? 131072 : (D * ESZ == 64 ? 49152 : 65536);
    static constexpr int NS = RING / STAGE;
    static constexpr int PITCH = D + 8;                            // floats per row of the merge buffer
    static constexpr int BUF = WK * M * PITCH * 4;
    static constexpr int SMEM = RING + BUF + 1024;
    static constexpr int BLOCKS_PER_SM = D == 256 ? 1 : 2;
};

struct SmallParams {
    AttnArgs a;
    CUtensorMap tk, tv;
    Partials part;
    int box_shift;                       // log2 of the rows of a TMA box
    int least;                           // smallest share, in steps
    long long wait_limit;
};

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two E4M3 codes (16 bits) -> two fp16
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t v) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(v));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <int D, bool F8, int WM>
__global__ void __launch_bounds__(SM_THREADS, (Small<D, F8, WM>::BLOCKS_PER_SM)) small_kernel(
    const __grid_constant__ SmallParams p) {
    using S = Small<D, F8, WM>;
    constexpr int NS = S::NS, WK = S::WK, M = S::M, EPL = D / 32;
    constexpr Tiling G{M, S::SK};
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    __shared__ ScanShared scan;
    __shared__ uint64_t full[NS], empty[NS];
    __shared__ uint32_t valid[NS];       // keys of the chunk that were loaded
    __shared__ float ml[WK * M][2];
    __shared__ int s_abort, s_stop;
    unsigned char* ring = sm_raw + ((1024 - (ptx::smem_u32(sm_raw) & 1023)) & 1023);
    float* buf = reinterpret_cast<float*>(ring + S::RING);
    volatile int* abort_flag = &s_abort;
    const AttnArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int i = 0; i < NS; ++i) {
            ptx::mbar_init(&full[i], 1);
            ptx::mbar_init(&empty[i], WM);
        }
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&p.tk);
        ptx::prefetch_tmap(&p.tv);
    }
    long long before;
    int b0, b1;
    const long long W = scan_steps(a, G, scan, &before, &b0, &b1);         // (synchronises)
    const int shares = W > 0 ? share_count(W, gridDim.x, p.least) : 0;
    if (threadIdx.x == 0) p.part.items[blockIdx.x].parts = 0;
    if (static_cast<int>(blockIdx.x) >= shares) return;
    const long long x0 = share_begin(W, blockIdx.x, shares), x1 = share_begin(W, blockIdx.x + 1, shares);
    Cursor cur = seek(a, G, scan, x0, before, b0, b1);
    long long left = x1 - x0;

    if (warp == 4) {
        // ------------------------------------------------------------ producer
        const int box = 1 << p.box_shift, pieces = CK >> p.box_shift;
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        while (left > 0 && ok) {
            const int lo = cur.step, hi = static_cast<int>(min(static_cast<long long>(cur.steps), lo + left));
            const int keys = tile_keys(a, cur.s, cur.mt, M);
            const int32_t* table = a.c.page_table + static_cast<size_t>(cur.b) * a.c.max_pages;
            // lane l holds the page of piece base + l; the next 32 are fetched ahead
            const int first = lo * S::SK, stop = min(hi * S::SK, keys);
            auto fetch = [&](int piece) {
                const int c = first + ((piece + lane) << p.box_shift);
                return c < stop ? table[c >> a.c.page_shift] : -1;
            };
            int base = 0;
            int page_now = fetch(0), page_next = fetch(32);
            for (int chunk = lo * WK; chunk < hi * WK && ok; ++chunk) {
                const int c0 = chunk * CK;
                const int at = (c0 - first) >> p.box_shift;
                if (at - base >= 32) {
                    base += 32;
                    page_now = page_next;
                    page_next = fetch(base + 32);
                }
                const int pg0 = __shfl_sync(0xFFFFFFFFu, page_now, (at - base) & 31);
                const int pg1 = __shfl_sync(0xFFFFFFFFu, page_now, (at - base + 1) & 31);
                if (lane == 0) {
                    ok = ptx::mbar_wait(&empty[stage], phase ^ 1u, abort_flag, p.wait_limit, a.status, 1u);
                    if (ok) {
                        uint32_t v = 0;
                        bool good[2] = {false, false};
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int c = c0 + q * box;
                            if (q >= pieces || c >= keys) continue;
                            const int pg = q ? pg1 : pg0;
                            good[q] = pg >= 0 && pg < a.c.num_pages;
                            if (!good[q]) report(a.status, MOE_ERR_DEVICE, cur.b);
                            else v |= (box == 32 ? 0xFFFFFFFFu : 0xFFFFu) << (q * 16);
                        }
                        const int rest = keys - c0;
                        if (rest < 32) v &= rest <= 0 ? 0u : (1u << rest) - 1u;
                        valid[stage] = v;
                        const uint32_t bytes = (static_cast<uint32_t>(good[0]) + good[1]) * 2u * box * D * S::ESZ;
                        ptx::mbar_arrive_expect_tx(&full[stage], bytes);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            if (!good[q]) continue;
                            unsigned char* dst = ring + stage * S::STAGE + q * box * D * S::ESZ;
                            const int slot = (c0 + q * box) & ((1 << a.c.page_shift) - 1), pg = q ? pg1 : pg0;
                            ptx::tma_load_5d(dst, &p.tk, &full[stage], 0, slot, 0, cur.h, pg);
                            ptx::tma_load_5d(dst + S::KBYTES, &p.tv, &full[stage], 0, slot, 0, cur.h, pg);
                        }
                    }
                }
                ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                if (++stage == NS) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
            left -= hi - lo;
            if (left > 0) cur.next(a, G);
        }
        if (lane == 0 && *abort_flag) {
            // every copy in flight lands before the block's memory goes away: stages below
            // `stage` were armed in this round, the others in the one before, if ever
            for (int i = 0; i < NS; ++i) {
                const uint32_t par = i < stage ? phase : phase ^ 1u;
                const long long t0 = clock64();
                while (!ptx::mbar_try_wait(&full[i], par) && clock64() - t0 < p.wait_limit) {
                }
            }
        }
        return;
    }

    // ---------------------------------------------------------------- compute warps
    const int wm = warp % WM, wk = warp / WM;
    const int g = lane >> 2, t = lane & 3;
    const int box = 1 << p.box_shift;
    const uint32_t ring_u = ptx::smem_u32(ring);
    const bool flip = a.scale_log2 < 0.f;                          // a negative scale: q changes sign instead
    const float scale = fabsf(a.scale_log2);
    // swizzled addresses: row r of a piece begins at r * ROWB, its 16-byte chunk c lies at c ^ f(r)
    auto row_off = [&](int key) {
        return (key >> p.box_shift) * (box * D * S::ESZ) + (key & (box - 1)) * S::ROWB;
    };
    auto swz = [&](int key) { return S::ROWB == 128 ? (key & 7) << 4 : ((key >> 1) & 3) << 4; };
    const int span_b = box * S::ROWB;                              // bytes between the spans of a row

    uint32_t chunk_no = wk;                                        // of this block, as the producer counts
    while (left > 0) {
        const int lo = cur.step, hi = static_cast<int>(min(static_cast<long long>(cur.steps), lo + left));
        const SeqInfo s = cur.s;
        const int rows = s.n * a.group;
        const int keys = tile_keys(a, s, cur.mt, M);
        const int r0 = cur.mt * M + wm * 16 + g;                   // this thread's rows: r0, r0 + 8
        const int i0 = min(r0, rows - 1) / a.group, i1 = min(r0 + 8, rows - 1) / a.group;

        // ---- Q as the first product's A operand
        uint32_t qf[D / 16][4];
        float sc0 = scale, sc1 = scale;
        {
            const uint32_t sign = flip ? 0x80008000u : 0u;
            const uint16_t* q0 = a.q + (s.row0 + i0) * a.q_stride + static_cast<long long>(cur.h * a.group + min(r0, rows - 1) % a.group) * D;
            const uint16_t* q1 = a.q + (s.row0 + i1) * a.q_stride + static_cast<long long>(cur.h * a.group + min(r0 + 8, rows - 1) % a.group) * D;
            const bool v0 = r0 < rows, v1 = r0 + 8 < rows;
            if constexpr (!F8) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int d = k * 16 + e * 8 + 2 * t;
                        qf[k][2 * e] = v0 ? *reinterpret_cast<const uint32_t*>(q0 + d) ^ sign : 0u;
                        qf[k][2 * e + 1] = v1 ? *reinterpret_cast<const uint32_t*>(q1 + d) ^ sign : 0u;
                    }
                }
            } else {
                // dimensions 32 blk + 8 t + 4 step + {0, 1 | 2, 3} stand for k = 2t, 2t+1 | 2t+8, 2t+9
                float m0 = 0.f, m1 = 0.f;
#pragma unroll
                for (int blk = 0; blk < D / 32; ++blk) {
                    uint4 x = make_uint4(0, 0, 0, 0), y = x;
                    if (v0) x = *reinterpret_cast<const uint4*>(q0 + blk * 32 + 8 * t);
                    if (v1) y = *reinterpret_cast<const uint4*>(q1 + blk * 32 + 8 * t);
                    qf[2 * blk][0] = x.x ^ sign; qf[2 * blk][2] = x.y ^ sign;
                    qf[2 * blk + 1][0] = x.z ^ sign; qf[2 * blk + 1][2] = x.w ^ sign;
                    qf[2 * blk][1] = y.x ^ sign; qf[2 * blk][3] = y.y ^ sign;
                    qf[2 * blk + 1][1] = y.z ^ sign; qf[2 * blk + 1][3] = y.w ^ sign;
                }
                auto amax = [](float m, uint32_t w) {
                    const float u = fabsf(__uint_as_float(w << 16)), v = fabsf(__uint_as_float(w & 0xFFFF0000u));
                    m = u < INFINITY ? fmaxf(m, u) : m;
                    return v < INFINITY ? fmaxf(m, v) : m;
                };
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    m0 = amax(amax(m0, qf[k][0]), qf[k][2]);
                    m1 = amax(amax(m1, qf[k][1]), qf[k][3]);
                }
#pragma unroll
                for (int o = 1; o < 4; o <<= 1) {
                    m0 = fmaxf(m0, __shfl_xor_sync(0xFFFFFFFFu, m0, o));
                    m1 = fmaxf(m1, __shfl_xor_sync(0xFFFFFFFFu, m1, o));
                }
                const int e0 = f16_chunk_exp(m0), e1 = f16_chunk_exp(m1);
                const float d0 = exp2_int(-e0), d1 = exp2_int(-e1);
                sc0 *= exp2_int(e0);
                sc1 *= exp2_int(e1);
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float d = (e & 1) ? d1 : d0;
                        qf[k][e] = pack_f16x2(__uint_as_float(qf[k][e] << 16) * d,
                                              __uint_as_float(qf[k][e] & 0xFFFF0000u) * d);
                    }
            }
        }

        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        bool ok = true;
        for (int st = lo; st < hi; ++st, chunk_no += WK) {
            const int stage = chunk_no % NS;
            ok = ptx::mbar_wait(&full[stage], (chunk_no / NS) & 1u, abort_flag, p.wait_limit, a.status, 2u);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const uint32_t vm = valid[stage];
            const int c0 = (st * WK + wk) * CK;
            if (vm != 0) {
                const uint32_t kb = ring_u + stage * S::STAGE, vb = kb + S::KBYTES;
                float sacc[4][4];
#pragma unroll
                for (int n = 0; n < 4; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sacc[n][e] = 0.f;
                if constexpr (!F8) {
                    const int krow = ((lane >> 4) << 3) + (lane & 7), kcol = ((lane >> 3) & 1) << 4;
                    const uint32_t ka0 = kb + row_off(krow), ka1 = kb + row_off(krow + 16);
                    const int x = swz(krow);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const int col = ((k & 3) * 32 + kcol) ^ x;
                        const uint32_t off = (k >> 2) * span_b + col;
                        uint32_t r[4];
                        ldsm4(r, ka0 + off);
                        mma16816<false>(sacc[0], qf[k], r[0], r[1]);
                        mma16816<false>(sacc[1], qf[k], r[2], r[3]);
                        ldsm4(r, ka1 + off);
                        mma16816<false>(sacc[2], qf[k], r[0], r[1]);
                        mma16816<false>(sacc[3], qf[k], r[2], r[3]);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const int key = n * 8 + g;
                        const uint32_t ka = kb + row_off(key);
                        const int x = swz(key);
#pragma unroll
                        for (int blk = 0; blk < D / 32; ++blk) {
                            const int byte = blk * 32 + 8 * t;
                            const uint32_t off = (byte / S::ROWB) * span_b + ((byte % S::ROWB) ^ x);
                            uint32_t w0, w1;
                            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w0), "=r"(w1) : "r"(ka + off) : "memory");
                            mma16816<true>(sacc[n], qf[2 * blk], e4m3x2_to_f16x2(w0), e4m3x2_to_f16x2(w0 >> 16));
                            mma16816<true>(sacc[n], qf[2 * blk + 1], e4m3x2_to_f16x2(w1), e4m3x2_to_f16x2(w1 >> 16));
                        }
                    }
                }
                // ---- scores in base 2, what a row does not see at -infinity
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    sacc[n][0] *= sc0;
                    sacc[n][1] *= sc0;
                    sacc[n][2] *= sc1;
                    sacc[n][3] *= sc1;
                }
                if (vm != 0xFFFFFFFFu || c0 + CK > s.ctx) {
                    const uint32_t see0 = seen_bits(a, s, i0, c0, keys) & vm, see1 = seen_bits(a, s, i1, c0, keys) & vm;
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int bit = n * 8 + 2 * t + e;
                            if (!(see0 >> bit & 1)) sacc[n][e] = -INFINITY;
                            if (!(see1 >> bit & 1)) sacc[n][2 + e] = -INFINITY;
                        }
                }
                float x0m = fmaxf(sacc[0][0], sacc[0][1]), x1m = fmaxf(sacc[0][2], sacc[0][3]);
#pragma unroll
                for (int n = 1; n < 4; ++n) {
                    x0m = fmaxf(x0m, fmaxf(sacc[n][0], sacc[n][1]));
                    x1m = fmaxf(x1m, fmaxf(sacc[n][2], sacc[n][3]));
                }
#pragma unroll
                for (int off = 1; off < 4; off <<= 1) {
                    x0m = fmaxf(x0m, __shfl_xor_sync(0xFFFFFFFFu, x0m, off));
                    x1m = fmaxf(x1m, __shfl_xor_sync(0xFFFFFFFFu, x1m, off));
                }
                const bool up0 = x0m > m0 + 8.f || (m0 == -INFINITY && x0m > m0);
                const bool up1 = x1m > m1 + 8.f || (m1 == -INFINITY && x1m > m1);
                if (__any_sync(0xFFFFFFFFu, up0 || up1)) {
                    const float n0 = up0 ? x0m : m0, n1 = up1 ? x1m : m1;
                    const float f0 = up0 ? ex2(m0 - n0) : 1.f, f1 = up1 ? ex2(m1 - n1) : 1.f;
                    m0 = n0;
                    m1 = n1;
                    l0 *= f0;
                    l1 *= f1;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][0] *= f0;
                        o[n][1] *= f0;
                        o[n][2] *= f1;
                        o[n][3] *= f1;
                    }
                }
                const float ref0 = m0 == -INFINITY ? 0.f : m0, ref1 = m1 == -INFINITY ? 0.f : m1;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    sacc[n][0] = ex2(sacc[n][0] - ref0);
                    sacc[n][1] = ex2(sacc[n][1] - ref0);
                    sacc[n][2] = ex2(sacc[n][2] - ref1);
                    sacc[n][3] = ex2(sacc[n][3] - ref1);
                    l0 += sacc[n][0] + sacc[n][1];
                    l1 += sacc[n][2] + sacc[n][3];
                }
                // ---- O += P V
                const int vrow = (((lane >> 3) & 1) << 3) + (lane & 7), vcol = (lane >> 4) << 4;
                const int xv = swz(vrow);
#pragma unroll
                for (int kp = 0; kp < 2; ++kp) {
                    uint32_t pf[4];
                    if constexpr (F8) {
                        pf[0] = pack_f16x2(sacc[2 * kp][0], sacc[2 * kp][1]);
                        pf[1] = pack_f16x2(sacc[2 * kp][2], sacc[2 * kp][3]);
                        pf[2] = pack_f16x2(sacc[2 * kp + 1][0], sacc[2 * kp + 1][1]);
                        pf[3] = pack_f16x2(sacc[2 * kp + 1][2], sacc[2 * kp + 1][3]);
                    } else {
                        pf[0] = pack_bf16x2(sacc[2 * kp][0], sacc[2 * kp][1]);
                        pf[1] = pack_bf16x2(sacc[2 * kp][2], sacc[2 * kp][3]);
                        pf[2] = pack_bf16x2(sacc[2 * kp + 1][0], sacc[2 * kp + 1][1]);
                        pf[3] = pack_bf16x2(sacc[2 * kp + 1][2], sacc[2 * kp + 1][3]);
                    }
                    // keys without a value in shared memory count as zero, not as 0 * whatever lies there
                    const uint32_t vk = vm >> (kp * 16 + 2 * t);
                    const uint32_t keep0 = ((vk & 1) ? 0xFFFFu : 0u) | ((vk & 2) ? 0xFFFF0000u : 0u);
                    const uint32_t keep1 = ((vk & 256) ? 0xFFFFu : 0u) | ((vk & 512) ? 0xFFFF0000u : 0u);
                    const uint32_t va = vb + row_off(kp * 16 + vrow);
                    if constexpr (!F8) {
#pragma unroll
                        for (int n = 0; n < D / 16; ++n) {
                            uint32_t r[4];
                            ldsm4_t(r, va + (n >> 2) * span_b + (((n & 3) * 32 + vcol) ^ xv));
                            if (vm != 0xFFFFFFFFu) {
                                r[0] &= keep0; r[1] &= keep1; r[2] &= keep0; r[3] &= keep1;
                            }
                            mma16816<false>(o[2 * n], pf, r[0], r[1]);
                            mma16816<false>(o[2 * n + 1], pf, r[2], r[3]);
                        }
                    } else {
#pragma unroll
                        for (int blk = 0; blk < D / 32; ++blk) {
                            const int byte = blk * 32;
                            uint32_t r[4];
                            ldsm4_t(r, va + (byte / S::ROWB) * span_b + (((byte % S::ROWB) + vcol) ^ xv));
                            if (vm != 0xFFFFFFFFu) {
                                r[0] &= keep0; r[1] &= keep1; r[2] &= keep0; r[3] &= keep1;
                            }
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t u = __byte_perm(r[2 * e], 0, 0x3120), v = __byte_perm(r[2 * e + 1], 0, 0x3120);
                                mma16816<true>(o[4 * blk + 2 * e], pf, e4m3x2_to_f16x2(u), e4m3x2_to_f16x2(v));
                                mma16816<true>(o[4 * blk + 2 * e + 1], pf, e4m3x2_to_f16x2(u >> 16), e4m3x2_to_f16x2(v >> 16));
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&empty[stage]);
        }

        // ---- the warps' results meet in shared memory
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, off);
            l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, off);
        }
        const int br = wk * M + wm * 16 + g;                       // row of the merge buffer
        if (t == 0) {
            ml[br][0] = m0;
            ml[br][1] = l0;
            ml[br + 8][0] = m1;
            ml[br + 8][1] = l1;
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float* dst = buf + (br + 8 * e) * S::PITCH;
            if constexpr (!F8) {
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
                    *reinterpret_cast<float2*>(dst + n * 8 + 2 * t) = make_float2(o[n][2 * e], o[n][2 * e + 1]);
            } else {
#pragma unroll
                for (int n = 0; n < D / 16; ++n)
                    *reinterpret_cast<float4*>(dst + n * 16 + 4 * t) =
                        make_float4(o[2 * n][2 * e], o[2 * n + 1][2 * e], o[2 * n][2 * e + 1], o[2 * n + 1][2 * e + 1]);
            }
        }
        compute_sync();
        const bool whole = lo == 0 && hi == cur.steps;
        const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (lo == 0);
        if (threadIdx.x == 0 && lo == 0 && !whole)                 // (the last of the share, so left == hi)
            p.part.items[blockIdx.x] = JoinItem{parts_until(W, shares, blockIdx.x, x1 - hi + cur.steps), s.row0, rows, cur.h, cur.mt};
        for (int r = warp; r < M; r += 4) {
            const int rr = cur.mt * M + r;
            if (rr >= rows) break;
            float m = ml[r][0];
#pragma unroll
            for (int w = 1; w < WK; ++w) m = fmaxf(m, ml[w * M + r][0]);
            float l = 0.f, acc[EPL];
#pragma unroll
            for (int j = 0; j < EPL; ++j) acc[j] = 0.f;
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int w = 0; w < WK; ++w) {
                const float f = ex2(ml[w * M + r][0] - ref);
                l += ml[w * M + r][1] * f;
#pragma unroll
                for (int j = 0; j < EPL; ++j) acc[j] += buf[(w * M + r) * S::PITCH + lane * EPL + j] * f;
            }
            const int i = rr / a.group, head = cur.h * a.group + rr % a.group;
            const long long row = s.row0 + i;
            bool nan = false;
#pragma unroll
            for (int j = 0; j < EPL; ++j) nan |= acc[j] != acc[j];
            if (hi * S::SK > s.ctx && l == l && __any_sync(0xFFFFFFFFu, nan)) {
                // 0 * infinity or NaN: a value that this row may not see; again, key by key
                float q[EPL];
#pragma unroll
                for (int j = 0; j < EPL; ++j) {
                    q[j] = bf16_to_f32(a.q[row * a.q_stride + head * D + lane * EPL + j]);
                    acc[j] = 0.f;
                }
                m = -INFINITY;
                l = 0.f;
                attend_row<EPL, F8>(a, cur.b, s, i, cur.h, q, lo * S::SK, min(hi * S::SK, keys), m, l, acc, lane);
            }
            if (whole) {
                const float inv = l == 0.f ? 0.f : a.c.v_scale / l;
                uint32_t w[EPL / 2];
#pragma unroll
                for (int j = 0; j < EPL; j += 2)
                    w[j / 2] = l == 0.f ? 0u : pack_bf16x2(acc[j] * inv, acc[j + 1] * inv);
                uint16_t* dst = a.out + row * a.out_stride + head * D + lane * EPL;
                if constexpr (EPL == 2) *reinterpret_cast<uint32_t*>(dst) = w[0];
                else if constexpr (EPL == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
                else *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[EPL / 2 - 2], w[EPL / 2 - 1]);
                if (a.lse != nullptr && lane == 0)
                    a.lse[row * a.n_q + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2F;
            } else {
                float* dst = p.part.o + (slot * M + r) * D + lane * EPL;
#pragma unroll
                for (int j = 0; j < EPL; ++j) dst[j] = acc[j];
                if (lane == 0) *reinterpret_cast<float2*>(p.part.ml + (slot * M + r) * 2) = make_float2(m, l);
            }
        }
        // after a wait that ran out every warp leaves here, at the same item
        if (threadIdx.x == 0) s_stop = *abort_flag;
        compute_sync();                                            // (and the merge buffer is free)
        if (s_stop) break;
        left -= hi - lo;
        if (left > 0) cur.next(a, G);
    }
}

template <int D, bool F8, int WM>
cudaError_t launch_cfg(const AttnArgs& a, void* partials, int sms, cudaStream_t st) {
    using S = Small<D, F8, WM>;
    SmallParams p;
    p.a = a;
    const int page = 1 << a.c.page_shift;
    const int box = page < CK ? page : CK;
    p.box_shift = page < CK ? a.c.page_shift : 5;
    p.least = 2;
    p.wait_limit = 4ll << 30;
    if (!make_kv_map(&p.tk, a, false, box, true) || !make_kv_map(&p.tv, a, true, box, true)) return cudaErrorInvalidValue;
    const int blocks = sms * S::BLOCKS_PER_SM < kSmallBlocks ? sms * S::BLOCKS_PER_SM : kSmallBlocks;
    p.part = partials_at(partials, blocks, S::M);
    const cudaError_t e = cudaFuncSetAttribute(small_kernel<D, F8, WM>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    {
        ProfileScope ps("tree_attention", st);
        small_kernel<D, F8, WM><<<blocks, SM_THREADS, S::SMEM, st>>>(p);
        note_launch();
    }
    const cudaError_t le = cudaGetLastError();
    if (le != cudaSuccess) return le;
    return launch_tree_attn_join(a, S::M, p.part, blocks, st);
}

template <int D, bool F8>
cudaError_t launch_d(const AttnArgs& a, void* partials, int sms, cudaStream_t st) {
    // rows of a tile: the smallest that holds a sequence's rows
    const long long rows = static_cast<long long>(a.c.max_new) * a.group;
    if (rows <= 16) return launch_cfg<D, F8, 1>(a, partials, sms, st);
    if (rows <= 32) return launch_cfg<D, F8, 2>(a, partials, sms, st);
    return launch_cfg<D, F8, 4>(a, partials, sms, st);
}

}  // namespace

cudaError_t launch_tree_attn_small(const AttnArgs& a, void* partials, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (sms <= 0) sms = 148;
    if (a.head_dim == 64) return a.f8 ? launch_d<64, true>(a, partials, sms, st) : launch_d<64, false>(a, partials, sms, st);
    if (a.head_dim == 128) return a.f8 ? launch_d<128, true>(a, partials, sms, st) : launch_d<128, false>(a, partials, sms, st);
    return a.f8 ? launch_d<256, true>(a, partials, sms, st) : launch_d<256, false>(a, partials, sms, st);
}

}  // namespace sre
