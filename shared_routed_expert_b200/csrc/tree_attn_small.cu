// Attention over a paged cache for few query rows per kv head (decoding, short drafts):
// bound by reading the cache once.
//
// Flash decoding with warp-level matrix instructions: a block takes tiles of M = 16
// or 32 packed query rows and runs along its share of the key axis (tree_attn.cuh). Its 8
// warps form 8 / WM groups of WM warps; the groups take chunks of CK keys in turn, each
// warp 16 rows, with its own running maximum and sum, so groups meet only at the end of an
// item. Each group has a ring of its own in shared memory that its first warp fills by TMA
// (one box per page piece and 128-byte span), K and V apart: the next K is on its way as
// soon as the scores are formed. Scores and the output accumulate in fp32 registers
// (m16n8k16); P is rounded to 16 bits as the second product's operand. What a warp does for
// a chunk is one chain of dependent steps, so warps are what hides latency: two blocks of 8
// per SM, with Q in shared memory to leave a thread within 128 registers, and no warp spent
// on loads alone (two blocks of 4 warps and a loading warp, Q in registers: 158 us for 64
// decode rows of 96 heads over 544 MB of E4M3 cache, here 120 us; 223 us for 128 rows over
// 566 MB of bf16 cache). 64 decode rows of 96 heads of 128: bf16 6.1 TB/s (1.09 GB in 180 us),
// E4M3 4.5 TB/s (4.3 back to back at the power limit), bound by the chain of a chunk (conversions, two products, exponentials) in
// 16 warps (chunks of half as many keys: 152 us). Heads of 64: 5.9 TB/s, of 256: 6.0 TB/s.
//   bf16 cache: Q, K, P, V as bf16.
//   E4M3 cache: K and V codes convert to fp16 exactly; Q rows are scaled by a power of two
//   to fp16 (exact for everything within 2^-28 of the row's largest entry) and P is fp16.
//   K's dimensions are taken in the order that lets a thread read 8 consecutive codes,
//   and V's 16-bit transposed loads return pairs of neighbouring dimensions that a byte
//   permutation turns into pairs of keys.
// The accumulators are rescaled only when a row's maximum grows by more than 2^8 (P stays
// below 2^8, or 2^15 over E4M3 caches, where fp16's range is used from its upper end: kLift).
#include "kernels.cuh"
#include "tc_ptx.cuh"
#include "tree_attn.cuh"

namespace sre {

namespace {

constexpr int NW = 8;                    // compute warps
constexpr int SM_THREADS = 32 * NW;

template <int D, bool F8, int WM>
struct Small {
    static constexpr int ESZ = F8 ? 1 : 2;
    // keys per chunk: 32 where a group's ring holds K and V of that many
    static constexpr int CK = WM == 1 && D * ESZ >= (D == 256 ? 512 : 256) ? 16 : 32;
    static constexpr int M = 16 * WM, WK = NW / WM, SK = CK * WK;
    static constexpr int ROWB = D * ESZ < 128 ? D * ESZ : 128;     // bytes of a row within one swizzle span
    static constexpr int SPANS = D * ESZ / ROWB;
    static constexpr int SPAN = CK * ROWB;                         // a chunk is stored [span][key][ROWB], swizzled
    static constexpr int KBYTES = SPANS * SPAN;                    // K (or V) of a chunk
    static constexpr int RING = D == 256 ? 131072 : 65536;
    static constexpr int NG = RING / (WK * 2 * KBYTES) < 4 ? RING / (WK * 2 * KBYTES) : 4;   // chunks a group holds
    static_assert(NG >= 1, "a group's ring holds a chunk");
    static constexpr int EXTRA = 2;                  // what an item costs besides its steps, in steps
    static constexpr int PITCH = D + 8;                            // floats per row of the merge buffer
    static constexpr int BUF = WK / 2 * M * PITCH * 4;             // half of the groups' results
    static constexpr int QPITCH = D * 2 + 16;                      // bytes per row of Q, which lies there before
    static_assert(M * QPITCH <= BUF, "Q fits the merge buffer");
    static constexpr int SMEM = RING + BUF + 1024;
    static constexpr int BLOCKS_PER_SM = D == 256 ? 1 : 2;
};

struct SmallParams {
    AttnArgs a;
    CUtensorMap tk, tv;
    Partials part;
    int box_shift;                       // log2 of the rows of a TMA box
    long long wait_limit;
    bool stall;                          // testing: no loads
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
__device__ __forceinline__ void compute_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// What a group loads of an item: its chunks start at key `first` and lie SK keys apart.
struct Chunks {
    const int32_t* table;
    int b, h, first, keys, n;
};

template <int D, bool F8, int WM>
__global__ void __launch_bounds__(SM_THREADS, (Small<D, F8, WM>::BLOCKS_PER_SM)) small_kernel(
    const __grid_constant__ SmallParams p) {
    using S = Small<D, F8, WM>;
    constexpr int WK = S::WK, M = S::M, EPL = D / 32, CK = S::CK, NG = S::NG;
    constexpr Tiling G{M, S::SK, S::EXTRA};
    constexpr uint32_t ALL = CK == 32 ? 0xFFFFFFFFu : 0xFFFFu;     // a chunk's keys as bits
    extern __shared__ __align__(1024) unsigned char sm_raw[];
    __shared__ ScanShared scan;
    __shared__ uint64_t kfull[WK][NG], vfull[WK][NG], kfree[WK][NG], vfree[WK][NG];
    __shared__ uint32_t valid[WK][NG];   // keys of the chunk that were loaded
    __shared__ float ml[NW * 16][2];
    __shared__ float q_scale[M];         // E4M3: what a row of Q was divided by, times the scale
    __shared__ int s_abort, s_stop, s_last;
    unsigned char* ring = sm_raw + ((1024 - (ptx::smem_u32(sm_raw) & 1023)) & 1023);
    float* buf = reinterpret_cast<float*>(ring + S::RING);
    unsigned char* q_smem = ring + S::RING;                        // (before the merge)
    volatile int* abort_flag = &s_abort;
    const AttnArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int i = 0; i < WK; ++i)
            for (int j = 0; j < NG; ++j) {
                ptx::mbar_init(&kfull[i][j], 1);
                ptx::mbar_init(&vfull[i][j], 1);
                ptx::mbar_init(&kfree[i][j], WM);
                ptx::mbar_init(&vfree[i][j], WM);
            }
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&p.tk);
        ptx::prefetch_tmap(&p.tv);
    }
    ScanThread me;
    const long long W = scan_units(a, G, scan, me);         // (synchronises)
    const Shares shares(W, gridDim.x, 1 + S::EXTRA);
    if (static_cast<int>(blockIdx.x) >= shares.count) return;
    const long long x0 = shares.begin(blockIdx.x), x1 = shares.begin(blockIdx.x + 1);
    Cursor cur = seek(a, G, scan, x0, me);
    long long left = x1 - x0;
    int lo, hi;
    if (!cur.segment(a, G, left, lo, hi)) return;

    const int wm = warp % WM, wk = warp / WM;
    const bool leads = wm == 0;
    const int g = lane >> 2, t = lane & 3;
    unsigned char* mem = ring + wk * NG * 2 * S::KBYTES;           // this group's ring: K, V, K, V, ...
    const uint32_t mem_u = ptx::smem_u32(mem);
    const bool flip = a.scale_log2 < 0.f;                          // a negative scale: q changes sign instead
    const float scale = fmaxf(fabsf(a.scale_log2), 1.0e-37f);      // (0 would turn what is not seen into NaN)
    // key k's row begins at k * ROWB of a span, its 16-byte chunk c lies at c ^ f(k)
    auto swz = [](int key) { return S::ROWB == 128 ? (key & 7) << 4 : ((key >> 1) & 3) << 4; };
    // where this lane's rows of the matrix loads begin in K and V, and the swizzle of their columns
    const int krow = F8 ? g : ((lane >> 4) << 3) + (lane & 7), vrow = (((lane >> 3) & 1) << 3) + (lane & 7);
    const uint32_t k_at = krow * S::ROWB, v_at = vrow * S::ROWB;
    const uint32_t k_x = F8 ? (8 * t) ^ swz(krow) : (((lane >> 3) & 1) << 4) ^ swz(krow), v_x = ((lane >> 4) << 4) ^ swz(vrow);

    // ---- loads, by the group's first warp
    const int box = 1 << p.box_shift, pieces = CK >> p.box_shift, batch = 32 / pieces;
    auto chunks_of = [&](const Cursor& c, int from, int to) {
        Chunks k;
        k.table = a.c.page_table + static_cast<size_t>(c.b) * a.c.max_pages;
        k.b = c.b;
        k.h = c.h;
        k.first = (from * WK + wk) * CK;
        k.keys = tile_keys(a, c.s, c.mt, M);
        const int stop = min(to * S::SK, k.keys);
        k.n = stop > k.first ? (stop - k.first + S::SK - 1) / S::SK : 0;
        return k;
    };
    // lane l has the page of piece l % pieces of chunk from + l / pieces
    auto fetch = [&](const Chunks& k, int from) {
        const int i = pieces == 1 ? from + lane : from + (lane >> 1);
        const int key = k.first + i * S::SK + (pieces == 1 ? 0 : (lane & 1) * box);
        return i < k.n && key < k.keys ? k.table[key >> a.c.page_shift] : -1;
    };
    int page_now = -1, page_next = -1, page_from = 0;              // of chunks page_from .. and the batch behind it
    uint32_t done = 0;                                             // chunks this group has finished
    // what is loaded of a chunk: pages of its pieces (-1: none), first key, bytes
    int pg[2] = {-1, -1}, at_key = 0;
    auto pages_of = [&](const Chunks& k, int i) {
        const int at = (i - page_from) * pieces;
        const int from = at < 32 ? page_now : page_next;
        at_key = k.first + i * S::SK;
        pg[0] = __shfl_sync(0xFFFFFFFFu, from, at & 31);
        if (static_cast<unsigned>(pg[0]) >= static_cast<unsigned>(a.c.num_pages)) {
            pg[0] = -1;
            if (lane == 0) report(a.status, MOE_ERR_DEVICE, k.b);
        }
        pg[1] = -1;
        if (pieces == 2) {
            pg[1] = __shfl_sync(0xFFFFFFFFu, from, (at + 1) & 31);
            if (static_cast<unsigned>(pg[1]) >= static_cast<unsigned>(a.c.num_pages)) {
                pg[1] = -1;
                if (at_key + box < k.keys && lane == 0) report(a.status, MOE_ERR_DEVICE, k.b);
            }
        }
    };
    // K (or V) of the chunk that pages_of looked at, the group's count-th; its stage has been read
    // once WM warps have freed it
    auto load = [&](const Chunks& k, uint32_t count, bool is_v) {
        if (lane == 0 && !p.stall) {
            const uint32_t st = count % NG;
            bool ok = true;
            if (WM > 1 && count >= NG)
                ok = ptx::mbar_wait(is_v ? &vfree[wk][st] : &kfree[wk][st], ((count / NG) - 1) & 1u, abort_flag, p.wait_limit,
                                    a.status, 1u);
            if (!is_v) {
                uint32_t v = ALL;
                if (pieces == 2) v = (pg[0] >= 0 ? 0xFFFFu : 0u) | (pg[1] >= 0 ? 0xFFFF0000u : 0u);
                else if (pg[0] < 0) v = 0;
                const int rest = k.keys - at_key;                  // >= 1
                if (rest < CK) v &= (1u << rest) - 1u;
                valid[wk][st] = v;
            }
            uint64_t* bar = is_v ? &vfull[wk][st] : &kfull[wk][st];
            if (ok) {
                ptx::mbar_arrive_expect_tx(bar, static_cast<uint32_t>((pg[0] >= 0) + (pg[1] >= 0)) * box * D * S::ESZ);
                unsigned char* dst = mem + (2 * st + is_v) * S::KBYTES;
                const int slot = at_key & ((1 << a.c.page_shift) - 1);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    if (pg[q] < 0) continue;
#pragma unroll
                    for (int sp = 0; sp < S::SPANS; ++sp)          // (a second piece is a page of its own)
                        ptx::tma_load_5d(dst + q * (CK / 2) * S::ROWB + sp * S::SPAN, is_v ? &p.tv : &p.tk, bar, 0, q ? 0 : slot, sp,
                                         k.h, pg[q]);
                }
            }
        }
        __syncwarp();
    };
    auto begin = [&](const Chunks& k) {
        page_from = 0;
        page_now = fetch(k, 0);
        page_next = k.n > batch ? fetch(k, batch) : -1;
        for (int i = 0; i < NG && i < k.n; ++i) {
            pages_of(k, i);
            load(k, done + i, false);
            load(k, done + i, true);
        }
    };
    Chunks ch = chunks_of(cur, lo, hi);
    if (leads) begin(ch);

    while (true) {
        const SeqInfo s = cur.s;
        const int rows = s.n * a.group;
        const int keys = ch.keys;
        const int r0 = cur.mt * M + wm * 16 + g;                   // this thread's rows: r0, r0 + 8
        const int i0 = token_of(a, min(r0, rows - 1)), i1 = token_of(a, min(r0 + 8, rows - 1));

        // ---- Q to shared memory: D / 8 lanes per row, 16 bytes each; rows behind the last are 0
        {
            constexpr int LPR = D / 8, RPI = NW * 32 / LPR, BATCH = (M + RPI - 1) / RPI;
            const uint32_t sign = flip ? 0x80008000u : 0u;
            const int ch = threadIdx.x % LPR;
            uint4 in[BATCH];                                       // all loads in flight before the stores
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int r = threadIdx.x / LPR + k * RPI, rr = cur.mt * M + r;
                in[k] = make_uint4(0, 0, 0, 0);
                if (r < M && rr < rows) {
                    const int i = token_of(a, rr);
                    in[k] = __ldg(reinterpret_cast<const uint4*>(
                        a.q + (s.row0 + i) * a.q_stride + static_cast<long long>(cur.h * a.group + rr - i * a.group) * D + ch * 8));
                }
            }
#pragma unroll
            for (int k = 0; k < BATCH; ++k) {
                const int r = threadIdx.x / LPR + k * RPI;
                const uint4 v = make_uint4(in[k].x ^ sign, in[k].y ^ sign, in[k].z ^ sign, in[k].w ^ sign);
                if constexpr (!F8) {
                    if (r < M) *reinterpret_cast<uint4*>(q_smem + r * S::QPITCH + ch * 16) = v;
                } else {
                    // a power of two brings the row to fp16; dimensions 32 blk + 8 t + 4 step +
                    // {0, 1 | 2, 3} stand for k = 2t, 2t+1 | 2t+8, 2t+9 of step 2 blk + step
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    float mx = 0.f;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float x = fabsf(__uint_as_float(w[j] << 16)), y = fabsf(__uint_as_float(w[j] & 0xFFFF0000u));
                        mx = x < INFINITY ? fmaxf(mx, x) : mx;
                        mx = y < INFINITY ? fmaxf(mx, y) : mx;
                    }
#pragma unroll
                    for (int o = 1; o < LPR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
                    const int e = f16_chunk_exp(mx);
                    const float d = exp2_int(-e);
                    if (r < M) {
                        unsigned char* dst = q_smem + r * S::QPITCH + (ch >> 2) * 64 + (ch & 3) * 4;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            *reinterpret_cast<uint32_t*>(dst + (j >> 1) * 32 + (j & 1) * 16) =
                                pack_f16x2(__uint_as_float(w[j] << 16) * d, __uint_as_float(w[j] & 0xFFFF0000u) * d);
                        if (ch == 0) q_scale[r] = fmaxf(scale * exp2_int(e), 1.0e-37f);
                    }
                }
            }
        }
        compute_sync();
        const uint32_t qa = ptx::smem_u32(q_smem) + (wm * 16 + (lane & 15)) * S::QPITCH + (lane >> 4) * 16;
        float sc0 = scale, sc1 = scale;
        if constexpr (F8) {
            sc0 = q_scale[wm * 16 + g];
            sc1 = q_scale[wm * 16 + g + 8];
        }

        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;

        constexpr int NT = CK / 8;                                 // key tiles of a chunk
        bool ok = true;
        for (int k = 0; k < ch.n; ++k, ++done) {
            const uint32_t stage = done % NG, par = (done / NG) & 1u;
            ok = ptx::mbar_wait(&kfull[wk][stage], par, abort_flag, p.wait_limit, a.status, 2u);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            const uint32_t vm = valid[wk][stage];
            const int c0 = ch.first + k * S::SK;
            {
                const uint32_t kb = mem_u + 2 * stage * S::KBYTES, vb = kb + S::KBYTES;
                float sacc[NT][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) sacc[n][e] = 0.f;
                if constexpr (!F8) {
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        const uint32_t at = kb + k_at + (d >> 2) * S::SPAN + (((d & 3) * 32) ^ k_x);
                        uint32_t q[4], r[NT / 2][4];
                        ldsm4(q, qa + d * 32);
#pragma unroll
                        for (int n = 0; n < NT / 2; ++n) ldsm4(r[n], at + n * 16 * S::ROWB);
#pragma unroll
                        for (int n = 0; n < NT / 2; ++n) {
                            mma16816<false>(sacc[2 * n], q, r[n][0], r[n][1]);
                            mma16816<false>(sacc[2 * n + 1], q, r[n][2], r[n][3]);
                        }
                    }
                } else {
#pragma unroll
                    for (int blk = 0; blk < D / 32; ++blk) {
                        uint32_t q0[4], q1[4];
                        ldsm4(q0, qa + blk * 64);
                        ldsm4(q1, qa + blk * 64 + 32);
                        const uint32_t at = kb + k_at + (blk * 32 / S::ROWB) * S::SPAN + ((blk * 32 % S::ROWB) ^ k_x);
                        uint32_t w0[NT], w1[NT];
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                         : "=r"(w0[n]), "=r"(w1[n])
                                         : "r"(at + n * 8 * S::ROWB)
                                         : "memory");
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint2 c = e4m3x4_to_f16x4(w0[n]);
                            mma16816<true>(sacc[n], q0, c.x, c.y);
                        }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint2 c = e4m3x4_to_f16x4(w1[n]);
                            mma16816<true>(sacc[n], q1, c.x, c.y);
                        }
                    }
                }
                // K has been read: the next one
                __syncwarp();
                if constexpr (WM > 1) {
                    if (lane == 0) ptx::mbar_arrive(&kfree[wk][stage]);
                }
                if (leads && k + NG < ch.n) {
                    pages_of(ch, k + NG);
                    load(ch, done + NG, false);
                }
                // ---- what a row does not see at -infinity
                if (vm != ALL || c0 + CK > s.ctx) {
                    const uint32_t see0 = seen_bits(a, s, i0, c0, keys) & vm, see1 = seen_bits(a, s, i1, c0, keys) & vm;
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int bit = n * 8 + 2 * t + e;
                            if (!(see0 >> bit & 1)) sacc[n][e] = -INFINITY;
                            if (!(see1 >> bit & 1)) sacc[n][2 + e] = -INFINITY;
                        }
                }
                float x0m = fmaxf(sacc[0][0], sacc[0][1]), x1m = fmaxf(sacc[0][2], sacc[0][3]);
#pragma unroll
                for (int n = 1; n < NT; ++n) {
                    x0m = fmaxf(x0m, fmaxf(sacc[n][0], sacc[n][1]));
                    x1m = fmaxf(x1m, fmaxf(sacc[n][2], sacc[n][3]));
                }
#pragma unroll
                for (int off = 1; off < 4; off <<= 1) {
                    x0m = fmaxf(x0m, __shfl_xor_sync(0xFFFFFFFFu, x0m, off));
                    x1m = fmaxf(x1m, __shfl_xor_sync(0xFFFFFFFFu, x1m, off));
                }
                // (m0, m1: unscaled)
                const bool up0 = (x0m - m0) * sc0 > 8.f || (m0 == -INFINITY && x0m > m0);
                const bool up1 = (x1m - m1) * sc1 > 8.f || (m1 == -INFINITY && x1m > m1);
                if (__any_sync(0xFFFFFFFFu, up0 || up1)) {
                    const float n0 = up0 ? x0m : m0, n1 = up1 ? x1m : m1;
                    const float f0 = up0 ? fast_exp2((m0 - n0) * sc0) : 1.f, f1 = up1 ? fast_exp2((m1 - n1) * sc1) : 1.f;
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
                const float ref0 = m0 == -INFINITY ? 0.f : lifted<F8>(m0 * sc0), ref1 = m1 == -INFINITY ? 0.f : lifted<F8>(m1 * sc1);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    sacc[n][0] = fast_exp2(fmaf(sacc[n][0], sc0, -ref0));
                    sacc[n][1] = fast_exp2(fmaf(sacc[n][1], sc0, -ref0));
                    sacc[n][2] = fast_exp2(fmaf(sacc[n][2], sc1, -ref1));
                    sacc[n][3] = fast_exp2(fmaf(sacc[n][3], sc1, -ref1));
                    l0 += sacc[n][0] + sacc[n][1];
                    l1 += sacc[n][2] + sacc[n][3];
                }
                // ---- O += P V
                ok = ptx::mbar_wait(&vfull[wk][stage], par, abort_flag, p.wait_limit, a.status, 3u);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
#pragma unroll
                for (int kp = 0; kp < CK / 16; ++kp) {
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
                    const uint32_t va = vb + v_at + kp * 16 * S::ROWB;
                    if constexpr (!F8) {
#pragma unroll
                        for (int n = 0; n < D / 16; ++n) {
                            uint32_t r[4];
                            ldsm4_t(r, va + (n >> 2) * S::SPAN + (((n & 3) * 32) ^ v_x));
                            if (vm != ALL) {
                                r[0] &= keep0; r[1] &= keep1; r[2] &= keep0; r[3] &= keep1;
                            }
                            mma16816<false>(o[2 * n], pf, r[0], r[1]);
                            mma16816<false>(o[2 * n + 1], pf, r[2], r[3]);
                        }
                    } else {
#pragma unroll
                        for (int blk = 0; blk < D / 32; ++blk) {
                            uint32_t r[4];
                            ldsm4_t(r, va + (blk * 32 / S::ROWB) * S::SPAN + ((blk * 32 % S::ROWB) ^ v_x));
                            if (vm != ALL) {
                                r[0] &= keep0; r[1] &= keep1; r[2] &= keep0; r[3] &= keep1;
                            }
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint2 u = e4m3x4_to_f16x4(__byte_perm(r[2 * e], 0, 0x3120));
                                const uint2 v = e4m3x4_to_f16x4(__byte_perm(r[2 * e + 1], 0, 0x3120));
                                mma16816<true>(o[4 * blk + 2 * e], pf, u.x, v.x);
                                mma16816<true>(o[4 * blk + 2 * e + 1], pf, u.y, v.y);
                            }
                        }
                    }
                }
            }
            __syncwarp();
            if constexpr (WM > 1) {
                if (lane == 0) ptx::mbar_arrive(&vfree[wk][stage]);
            }
            if (leads) {
                if (k + NG < ch.n) load(ch, done + NG, true);
                if (k + 1 - page_from >= batch) {
                    page_from += batch;
                    page_now = page_next;
                    page_next = fetch(ch, page_from + batch);
                }
            }
        }
        // the next item's first chunks are on their way while this one's results are joined
        Cursor nxt = cur;
        Chunks nch = ch;
        long long nleft = left;
        int nlo = 0, nhi = 0;
        const bool more = ok && nxt.segment(a, G, nleft, nlo, nhi);
        if (more) {
            nch = chunks_of(nxt, nlo, nhi);
            if (leads) begin(nch);
        }

        // ---- the warps' results meet in shared memory, maxima in base 2
        m0 = lifted<F8>(m0 * sc0);
        m1 = lifted<F8>(m1 * sc1);
#pragma unroll
        for (int off = 1; off < 4; off <<= 1) {
            l0 += __shfl_xor_sync(0xFFFFFFFFu, l0, off);
            l1 += __shfl_xor_sync(0xFFFFFFFFu, l1, off);
        }
        constexpr int HK = WK / 2;
        auto spot = [&](int e, int n) {                            // this thread's places in rows g + 8e of its group's part
            float* dst = buf + ((wk % HK) * M + wm * 16 + g + 8 * e) * S::PITCH;
            return F8 ? dst + n * 16 + 4 * t : dst + n * 8 + 2 * t;
        };
        const int br = (wk % HK) * M + wm * 16 + g;
        compute_sync();                                            // Q has been read
#pragma unroll
        for (int round = 0; round < 2; ++round) {
            // the upper half of the groups leaves its results, the lower half adds its own
            if (round == 1) compute_sync();
            if ((round == 0) != (wk >= HK)) continue;
            float f0 = 1.f, f1 = 1.f, g0 = 0.f, g1 = 0.f;
            if (round == 1) {
                const float2 a0 = *reinterpret_cast<const float2*>(ml[br]), a1 = *reinterpret_cast<const float2*>(ml[br + 8]);
                const float n0 = fmaxf(m0, a0.x), n1 = fmaxf(m1, a1.x);
                const float ref0 = n0 == -INFINITY ? 0.f : n0, ref1 = n1 == -INFINITY ? 0.f : n1;
                f0 = fast_exp2(m0 - ref0);
                f1 = fast_exp2(m1 - ref1);
                g0 = fast_exp2(a0.x - ref0);
                g1 = fast_exp2(a1.x - ref1);
                m0 = n0;
                m1 = n1;
                l0 = l0 * f0 + a0.y * g0;
                l1 = l1 * f1 + a1.y * g1;
                __syncwarp();                                      // (the quad has read its row's statistics)
            }
            if (t == 0) {
                *reinterpret_cast<float2*>(ml[br]) = make_float2(m0, l0);
                *reinterpret_cast<float2*>(ml[br + 8]) = make_float2(m1, l1);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float f = e ? f1 : f0, gg = e ? g1 : g0;
                if constexpr (!F8) {
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        float2* at = reinterpret_cast<float2*>(spot(e, n));
                        float2 v = make_float2(o[n][2 * e], o[n][2 * e + 1]);
                        if (round == 1) {
                            const float2 u = *at;
                            v = make_float2(v.x * f + u.x * gg, v.y * f + u.y * gg);
                        }
                        *at = v;
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < D / 16; ++n) {
                        float4* at = reinterpret_cast<float4*>(spot(e, n));
                        float4 v = make_float4(o[2 * n][2 * e], o[2 * n + 1][2 * e], o[2 * n][2 * e + 1], o[2 * n + 1][2 * e + 1]);
                        if (round == 1) {
                            const float4 u = *at;
                            v = make_float4(v.x * f + u.x * gg, v.y * f + u.y * gg, v.z * f + u.z * gg, v.w * f + u.w * gg);
                        }
                        *at = v;
                    }
                }
            }
        }
        compute_sync();
        const bool whole = lo == 0 && hi == cur.steps;
        const size_t slot = 2 * static_cast<size_t>(blockIdx.x) + (lo == 0);
        for (int r = warp; r < M; r += NW) {
            const int rr = cur.mt * M + r;
            if (rr >= rows) break;
            float m = ml[r][0];
#pragma unroll
            for (int w = 1; w < HK; ++w) m = fmaxf(m, ml[w * M + r][0]);
            float l = 0.f, acc[EPL];
#pragma unroll
            for (int j = 0; j < EPL; ++j) acc[j] = 0.f;
            const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int w = 0; w < HK; ++w) {
                const float f = fast_exp2(ml[w * M + r][0] - ref);
                l += ml[w * M + r][1] * f;
#pragma unroll
                for (int j = 0; j < EPL; ++j) acc[j] += buf[(w * M + r) * S::PITCH + lane * EPL + j] * f;
            }
            const int i = token_of(a, rr), head = cur.h * a.group + rr - i * a.group;
            const long long row = s.row0 + i;
            bool nan = false;
#pragma unroll
            for (int j = 0; j < EPL; ++j) nan |= acc[j] != acc[j];
            if (hi * S::SK > s.ctx && l == l && __any_sync(0xFFFFFFFFu, nan) &&
                hides_infinities<D, F8>(a, cur.b, s, i, cur.h, lo * S::SK, min(hi * S::SK, keys), lane)) {
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
                const float inv = l == 0.f ? 0.f : __fdividef(a.c.v_scale, l);
                uint32_t w[EPL / 2];
#pragma unroll
                for (int j = 0; j < EPL; j += 2)
                    w[j / 2] = l == 0.f ? 0u : pack_bf16x2(acc[j] * inv, acc[j + 1] * inv);
                uint16_t* dst = a.out + row * a.out_stride + head * D + lane * EPL;
                if constexpr (EPL == 2) *reinterpret_cast<uint32_t*>(dst) = w[0];
                else if constexpr (EPL == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
                else *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[EPL / 2 - 2], w[EPL / 2 - 1]);
                if (a.lse != nullptr && lane == 0)
                    a.lse[row * a.n_q + head] = lse_of(m, l);
            } else {
                float* dst = p.part.o + (slot * M + r) * D + lane * EPL;
#pragma unroll
                for (int j = 0; j < EPL; ++j) dst[j] = acc[j];
                if (lane == 0) *reinterpret_cast<float2*>(p.part.ml + (slot * M + r) * 2) = make_float2(m, l);
            }
        }
        if (!whole) {
            // the last block to leave its part of the item joins them (one sequence of 4096 keys over 91
            // blocks, 8 parts' loads in flight: 16.7 us; 4: 18.0, 12: 15.9, but registers spill, and 64
            // sequences take 126 us instead of 120; finer shares make the join longer: 21 us with 272 blocks)
            const int2 in = item_shares(shares, cur, G, x1, left);
            compute_sync();
            if (threadIdx.x == 0) {
                unsigned before;                                   // (the barrier put the others' writes before it)
                asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(p.part.arrived + in.x) : "memory");
                const bool last = before == static_cast<unsigned>(in.y) - 1u;
                if (last) p.part.arrived[in.x] = 0;
                s_last = last;
            }
            compute_sync();
            if (s_last) {
                for (int r = warp; r < M && cur.mt * M + r < rows; r += NW)
                    join_row<EPL, 8>(a, p.part, M, in.x, in.y, s.row0, cur.h, r, cur.mt * M + r, lane);
            }
        }
        // after a wait that ran out every warp leaves here, at the same item
        if (threadIdx.x == 0) s_stop = *abort_flag;
        compute_sync();                                            // (and the merge buffer is free)
        if (s_stop || !more) break;
        cur = nxt;
        ch = nch;
        left = nleft;
        lo = nlo;
        hi = nhi;
    }
    if (s_stop && leads && lane == 0) {
        // loads in flight land before the block's memory goes away: the last use of each stage, if
        // it was not waited for, is the one `done` or the one NG - 1 chunks behind it at most
        for (uint32_t i = done; i < done + NG; ++i) {
            const long long t0 = clock64();
            while (!(ptx::mbar_try_wait(&kfull[wk][i % NG], (i / NG) & 1u) && ptx::mbar_try_wait(&vfull[wk][i % NG], (i / NG) & 1u)) &&
                   clock64() - t0 < (1ll << 24)) {
            }
        }
    }
}

template <int D, bool F8, int WM>
cudaError_t launch_cfg(const AttnArgs& a, void* partials, int sms, cudaStream_t st) {
    using S = Small<D, F8, WM>;
    SmallParams p;
    p.a = a;
    const int page = 1 << a.c.page_shift;
    const int box = page < S::CK ? page : S::CK;
    p.box_shift = page < S::CK ? a.c.page_shift : (S::CK == 32 ? 5 : 4);
    p.stall = tree_attn_take_stall();
    p.wait_limit = p.stall ? 20ll << 20 : 4ll << 30;
    if (!make_kv_map(&p.tk, a, false, box) || !make_kv_map(&p.tv, a, true, box)) return cudaErrorInvalidValue;
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
    return cudaSuccess;
}

template <int D, bool F8>
cudaError_t launch_d(const AttnArgs& a, void* partials, int sms, cudaStream_t st) {
    // rows of a tile: the smallest that holds a sequence's rows
    const long long rows = static_cast<long long>(a.c.max_new) * a.group;
    return rows <= 16 ? launch_cfg<D, F8, 1>(a, partials, sms, st) : launch_cfg<D, F8, 2>(a, partials, sms, st);
}

}  // namespace

// A block here has done its first chunk before the tiles of the other kernels have begun (they
// allocate TMEM, fill a pipeline of steps and have a second launch for the join), so a call that
// keeps each block busy for no more than a few units is done sooner here: 14 sequences of 21 to 65
// tokens of 10 heads over 2 kv heads, E4M3, 14 us here, 28 us there; 2 sequences of 49 and 149 tokens of
// 12 heads behind 1278 keys 24 and 39 us; 3 sequences of 266 to 800 tokens of 4 heads behind
// 1515 keys, 10 units a block, 60 us and 41 us there. The contexts are on the device; what the
// page table can hold bounds them, so a table much wider than its sequences (131072 tokens: 515 units)
// leaves no call but one of a tile or two short, and those drafts take the tiles' 28 us.
bool tree_attn_short(const AttnArgs& a) {
    const long long tiles = (static_cast<long long>(a.T) * a.group / 32 + a.c.B) * a.c.n_kv;
    const long long units = (static_cast<long long>(a.c.max_pages) << a.c.page_shift) / 256 + 3;
    return tiles * units <= 4 * 296;
}

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
