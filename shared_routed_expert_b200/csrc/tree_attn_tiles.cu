// Attention over a paged cache for many query rows per kv head (prefill chunks, larger
// trees): bound by the tensor cores and the exponentials.
//
// A block takes tiles of 256 packed query rows as two halves of 128 that take turns on the
// tensor cores, and runs along its share of the key axis (tree_attn.cuh) in steps of 128 keys:
//   S_h = Q_h K^T         tcgen05.mma, Q and K in shared memory, S in TMEM (fp32)
//   P_h = 2^(S_h - m)     four warps per half, one thread per row; P (bf16) overwrites S in TMEM
//   O_h += P_h V          tcgen05.mma with P read from TMEM, V in shared memory (keys as K,
//                         so V is used as it is stored, MN-major), O in TMEM (fp32)
// While one half's exponentials run, the other half's products do. The running maximum is
// raised (and O rescaled, in TMEM) only when a row's grows by more than 2^8, so that
// rescaling is rare; sums and statistics are fp32, P is rounded to bf16 for the product.
// A tile of no more than 128 rows (short drafts, the ends of sequences) has both halves work
// on the same rows, on every second step each, and the first half join the two sums.
// Roles: warps 0-3 and 4-7 the two halves' softmax, loads of Q and epilogue; warp 8 issues
// the products; warp 9 streams K and V boxes (one per page piece and 128-byte span) through
// a ring in shared memory. Every wait is bounded.
// Measured, 96 heads of 128 over 8 kv heads, bf16: a chunk of 4096 rows behind 12288 keys 2.72 to
// 2.85 ms, 1010 to 1060 TFLOP/s at the power limit of 1000 W (1.7 to 1.78 GHz); trees of 23 to 61 nodes
// of 12 sequences 185 us in short runs (740 TFLOP/s; the join is 13 us of it), 212 us back to back at
// the power limit (640 TFLOP/s, 1.74 GHz); 4-token chains of 32 sequences 107 us (5.3 TB/s) and 120 us
// (4.7 TB/s, 1.66 GHz).
// The exponentials of a half take about as long as its products (128 per thread and step). No
// faster for the chunk: the whole row of S in registers (2987 us, spills), a quartic in place of
// 1/8 to 3/8 of the exponentials (3004 to 3137 us), P in two arrivals (2909 us, one 2913 then),
// steps of 64 keys with two S (4950 us: a product of N = 64 takes as long as one of 128).
// E4M3 caches: the boxes go to a ring of codes, from which warps 10 and 11 write K and V as
// fp16 (exact) to the products' ring (2048 rows behind 8192 keys: 1110 us, bf16 870 to 940 us; the
// 4-token chains 175 us, the trees 256 us). Q rows are scaled by a power of two to fp16 (exact for
// everything within 2^-28 of the row's largest entry) and P is fp16, raised by 2^7 (kLift). (E4M3
// operands would need P in 4 significant bits.)
#include "kernels.cuh"
#include "tc_ptx.cuh"
#include "tree_attn.cuh"

namespace sre {

namespace {

constexpr int TK = 128;                  // keys per step
constexpr int TL_THREADS = 320, TL_THREADS_F8 = 384;
constexpr int kTileExtra = 4;            // what an item costs besides its steps, in steps (2: those chains 138 us)
// Rows of a kv head from which this kernel takes over. Above 32 rows each 16 of them cost the
// other kernel (tree_attn_small.cu) a pass over K and V in shared memory: 32 sequences of 4 rows
// of 96 heads (48 rows a kv head), 566 MB of bf16 cache: 107 us here, 195 us there.
constexpr int kTileLeastRows = 32;
// Units of the shortest share: with 8, 12 sequences of 30 to 90 tokens of 20 heads over 4 kv heads behind up
// to 153 keys, E4M3, take 40 us instead of 29
constexpr int kTileLeastShare = 3;
constexpr int kInfo = 8;                 // steps whose key masks are kept (the producer is at most 6 ahead)

template <int D, bool F8>
struct Tile {
    static constexpr int SPANS = D * 2 / 128;
    static constexpr int SPAN = 128 * 128;                         // bytes of a span of 128 rows
    static constexpr int QHALF = SPANS * SPAN;
    static constexpr int SLOT = SPANS * SPAN;                      // K or V of a step, 16 bits each
    static constexpr int NS = F8 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 10);
    static constexpr int CODES = TK * D;                           // K or V of a step as E4M3 codes
    static constexpr int NR = F8 ? 4 : 0;
    static constexpr int SMEM = 2 * QHALF + NS * SLOT + NR * CODES + 1024;
    // what is loaded by TMA, at the rows' own width
    static constexpr int ROWB = F8 ? D : 128;
    static constexpr int LOAD_SPANS = F8 ? 1 : SPANS, LOAD_SPAN = TK * ROWB;
};

struct TileParams {
    AttnArgs a;
    CUtensorMap tk, tv;
    Partials part;
    int box_shift;
    long long wait_limit;
    bool stall;                          // testing: no loads
};

template <int D, bool F8>
__global__ void __launch_bounds__(F8 ? TL_THREADS_F8 : TL_THREADS, 1) tiles_kernel(const __grid_constant__ TileParams p) {
    using S = Tile<D, F8>;
    constexpr int NS = S::NS, NR = S::NR > 0 ? S::NR : 1;
    constexpr Tiling G{kTileRows, TK, kTileExtra};
    extern __shared__ __align__(1024) unsigned char tl_raw[];
    __shared__ ScanShared scan;
    __shared__ uint64_t full[NS], empty[NS], q_ready[2], s_full[2], p_ready[2], o_full[2], x_ready, x_done, tail_bar, drain_bar;
    __shared__ uint64_t raw_full[NR], raw_free[NR];
    __shared__ float q_scale[2][128];    // E4M3: what a row of Q was divided by, times the scale
    __shared__ uint32_t info[kInfo][4];  // keys of a step that were loaded
    __shared__ uint32_t tmem_base_s;
    __shared__ int s_abort;
    unsigned char* smem = tl_raw + ((1024 - (ptx::smem_u32(tl_raw) & 1023)) & 1023);
    unsigned char* ring = smem + 2 * S::QHALF;
    unsigned char* codes = ring + NS * S::SLOT;
    // where both halves work on the same rows, the second half's maxima (base 2) and sums lie in its Q
    float2* x_ml = reinterpret_cast<float2*>(smem + S::QHALF);
    volatile int* abort_flag = &s_abort;
    const AttnArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int i = 0; i < NS; ++i) {
            ptx::mbar_init(&full[i], F8 ? 2 : 1);
            ptx::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NR; ++i) {
            ptx::mbar_init(&raw_full[i], 1);
            ptx::mbar_init(&raw_free[i], 2);
        }
        for (int h = 0; h < 2; ++h) {
            ptx::mbar_init(&q_ready[h], 128);
            ptx::mbar_init(&s_full[h], 1);
            ptx::mbar_init(&p_ready[h], 128);
            ptx::mbar_init(&o_full[h], 1);
        }
        ptx::mbar_init(&x_ready, 128);
        ptx::mbar_init(&x_done, 128);
        ptx::mbar_init(&tail_bar, 1);
        ptx::mbar_init(&drain_bar, 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&p.tk);
        ptx::prefetch_tmap(&p.tv);
    }
    ScanThread me;
    const long long W = scan_units(a, G, scan, me);
    const Shares shares(W, gridDim.x, kTileLeastShare);
    if (threadIdx.x == 0) p.part.items[blockIdx.x].parts = 0;
    if (static_cast<int>(blockIdx.x) >= shares.count) return;
    const long long x0 = shares.begin(blockIdx.x), x1 = shares.begin(blockIdx.x + 1);
    Cursor cur = seek(a, G, scan, x0, me);
    long long left = x1 - x0;
    int lo, hi;
    if (warp == 8) {
        ptx::tmem_alloc(&tmem_base_s, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_base_s;   // columns: S0 0, S1 128, O0 256, O1 384

    if (warp == 9) {
        // ------------------------------------------------------------ producer
        const int box = 1 << p.box_shift, pieces = TK >> p.box_shift;
        uint32_t n = 0, step_no = 0, tail_phase = 0;               // slots and steps so far
        bool ok = !p.stall;
        while (ok && cur.segment(a, G, left, lo, hi)) {
            const int keys = tile_keys(a, cur.s, cur.mt, G.M);
            const int32_t* table = a.c.page_table + static_cast<size_t>(cur.b) * a.c.max_pages;
            const int first = lo * TK, stop = min(hi * TK, keys);
            auto fetch = [&](int piece) {
                const int c = first + ((piece + lane) << p.box_shift);
                return c < stop ? table[c >> a.c.page_shift] : -1;
            };
            int base = 0;
            int page_now = fetch(0), page_next = fetch(32);
            for (int st = lo; st < hi && ok; ++st, ++step_no) {
                const int c0 = st * TK;
                const int at = (c0 - first) >> p.box_shift;
                if (at - base >= 32) {                             // (pieces per step divide 32)
                    base += 32;
                    page_now = page_next;
                    page_next = fetch(base + 32);
                }
                // lane q < pieces: piece q of this step
                const int page = __shfl_sync(0xFFFFFFFFu, page_now, (at - base + lane) & 31);
                const int c = c0 + (lane << p.box_shift);
                const bool wanted = lane < pieces && c < keys;
                const bool good = wanted && page >= 0 && page < a.c.num_pages;
                if (wanted && !good) report(a.status, MOE_ERR_DEVICE, cur.b);
                const uint32_t goods = __ballot_sync(0xFFFFFFFFu, good);
                uint32_t word = 0xFFFFFFFFu;                       // lane q < 4: keys 32 q .. of the step
                {
                    const int k0 = lane * 32, rest = keys - (c0 + k0);
                    if (rest < 32) word = rest <= 0 ? 0u : (1u << rest) - 1u;
                    if (box >= 32) {
                        if (!(goods >> ((k0 >> p.box_shift) & 31) & 1)) word = 0;
                    } else {
                        if (!(goods >> ((2 * lane) & 31) & 1)) word &= 0xFFFF0000u;
                        if (!(goods >> ((2 * lane + 1) & 31) & 1)) word &= 0xFFFFu;
                    }
                }
                if (lane < 4) info[step_no % kInfo][lane] = word;
                __syncwarp();
                const bool partial = __any_sync(0xFFFFFFFFu, lane < 4 && word != 0xFFFFFFFFu);
                const uint32_t bytes = static_cast<uint32_t>(__popc(goods)) * box * S::ROWB * S::LOAD_SPANS;
                const int slot_in_page = c & ((1 << a.c.page_shift) - 1);
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++n) {
                    const uint32_t sl = F8 ? n % NR : n % NS, use = F8 ? n / NR : n / NS;
                    ok = ok && ptx::mbar_wait(F8 ? &raw_free[sl] : &empty[sl], (use & 1u) ^ 1u, abort_flag, p.wait_limit, a.status, 1u);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const bool tail = !F8 && kv == 1 && partial;
                    uint64_t* bar = F8 ? &raw_full[sl] : (tail ? &tail_bar : &full[sl]);
                    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, bytes);
                    __syncwarp();
                    unsigned char* dst = F8 ? codes + sl * S::CODES : ring + sl * S::SLOT;
                    if (good) {
#pragma unroll
                        for (int sp = 0; sp < S::LOAD_SPANS; ++sp)
                            ptx::tma_load_5d(dst + sp * S::LOAD_SPAN + lane * box * S::ROWB, kv ? &p.tv : &p.tk, bar, 0, slot_in_page,
                                             sp, cur.h, page);
                    }
                    if (tail) {
                        // keys that are not there count as zero, not as 0 * whatever lies there
                        ok = ptx::mbar_wait(&tail_bar, tail_phase, abort_flag, p.wait_limit, a.status, 7u);
                        tail_phase ^= 1u;
                        ok = __all_sync(0xFFFFFFFFu, ok);
#pragma unroll 1
                        for (int r = lane; r < TK; r += 32) {
                            const uint32_t w = __shfl_sync(0xFFFFFFFFu, word, r >> 5);
                            if (w >> (r & 31) & 1) continue;
                            for (int sp = 0; sp < S::SPANS; ++sp)
#pragma unroll
                                for (int ch = 0; ch < 8; ++ch)
                                    *reinterpret_cast<uint4*>(dst + sp * S::SPAN + r * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
                        }
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&full[sl]);
                    }
                }
            }
        }
        if (lane == 0 && *abort_flag) {
            // every copy in flight lands before the block's memory goes away
            constexpr uint32_t kSlots = F8 ? NR : NS;
            for (uint32_t i = 0; i < kSlots; ++i) {
                const uint32_t uses = n > i ? (n - i + kSlots - 1) / kSlots : 0;   // times slot i was armed
                if (uses == 0) continue;
                const long long t0 = clock64();
                while (!ptx::mbar_try_wait(F8 ? &raw_full[i] : &full[i], (uses - 1) & 1u) && clock64() - t0 < p.wait_limit) {
                }
            }
        }
    } else if (warp == 8) {
        // ------------------------------------------------------------ products
        if (lane == 0) {
            constexpr uint32_t IS = ptx::instr_desc(128, TK, F8 ? 0 : 1);
            constexpr uint32_t IO = ptx::instr_desc(128, D, F8 ? 0 : 1) | ptx::kBMnMajor;
            const uint32_t q_u = ptx::smem_u32(smem), ring_u = ptx::smem_u32(ring);
            uint32_t n = 0, qp[2] = {0, 0}, pp[2] = {0, 0};
            bool ok = true;
            auto wait = [&](uint64_t* bar, uint32_t par, unsigned site) {
                ok = ok && ptx::mbar_wait(bar, par, abort_flag, p.wait_limit, a.status, site);
                return ok;
            };
            // descriptors differ in their start address alone (16-byte units in the low word)
            const uint64_t d_k = ptx::smem_desc_sw<128>(0), d_mn = ptx::smem_desc_mn128(0, S::SPAN);
            const uint32_t k_hi = static_cast<uint32_t>(d_k >> 32), k_lo = static_cast<uint32_t>(d_k);
            const uint32_t mn_hi = static_cast<uint32_t>(d_mn >> 32), mn_lo = static_cast<uint32_t>(d_mn);
            auto desc = [](uint32_t hi_w, uint32_t lo_w) { return static_cast<uint64_t>(hi_w) << 32 | lo_w; };
            auto scores = [&](int h, int qh, uint32_t kslot) {
                const uint32_t ka = k_lo + ((ring_u + kslot * S::SLOT) >> 4), qa = k_lo + ((q_u + qh * S::QHALF) >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * S::SPAN + (k & 3) * 32) >> 4;
                    ptx::mma_f16(tmem + h * 128, desc(k_hi, qa + off), desc(k_hi, ka + off), IS, k != 0);
                }
            };
            auto values = [&](int h, uint32_t vslot, bool add) {
                const uint32_t va = mn_lo + ((ring_u + vslot * S::SLOT) >> 4);
#pragma unroll
                for (int k = 0; k < TK / 16; ++k)
                    ptx::mma_f16_ts(tmem + 256 + h * 128, tmem + h * 128 + 64 + k * 8, desc(mn_hi, va + k * 128), IO, add || k != 0);
            };
            while (ok && cur.segment(a, G, left, lo, hi)) {
                const bool two = cur.s.n * a.group - cur.mt * G.M > 128;
                if (!two && hi - lo > 1) {
                    // half h takes steps lo + h, lo + h + 2, ... of the same rows
                    if (!wait(&q_ready[0], qp[0], 4u)) break;
                    qp[0] ^= 1u;
#pragma unroll 1
                    for (int st = lo - 2; st < hi; ++st) {
                        const int h = (st - lo) & 1;
                        const uint32_t kn = n + 2 * (st + 2 - lo), vn = n + 2 * (st - lo) + 1;
                        if (st >= lo) {
                            if (!wait(&full[vn % NS], (vn / NS) & 1u, 3u) || !wait(&p_ready[h], pp[h], 5u)) break;
                            pp[h] ^= 1u;
                            ptx::tc_fence_after();
                            values(h, vn % NS, st > lo + 1);
                            ptx::mma_commit(&empty[vn % NS]);
                            if (st + 2 >= hi) ptx::mma_commit(&o_full[h]);
                        }
                        if (st + 2 < hi) {
                            if (!wait(&full[kn % NS], (kn / NS) & 1u, 3u)) break;
                            ptx::tc_fence_after();
                            scores(h, 0, kn % NS);
                            ptx::mma_commit(&s_full[h]);
                            ptx::mma_commit(&empty[kn % NS]);
                        }
                    }
                    n += 2 * (hi - lo);
                    continue;
                }
                if (!wait(&full[n % NS], (n / NS) & 1u, 3u)) break;
#pragma unroll 1
                for (int h = 0; h < (two ? 2 : 1); ++h) {
                    if (!wait(&q_ready[h], qp[h], 4u)) break;
                    qp[h] ^= 1u;
                    ptx::tc_fence_after();
                    scores(h, h, n % NS);
                    ptx::mma_commit(&s_full[h]);
                }
                if (!ok) break;
                ptx::mma_commit(&empty[n % NS]);
                for (int st = lo; st < hi; ++st, n += 2) {
                    const bool more = st + 1 < hi;
                    const uint32_t vn = n + 1, kn = n + 2;
                    if (!wait(&full[vn % NS], (vn / NS) & 1u, 3u)) break;
#pragma unroll 1
                    for (int h = 0; h < (two ? 2 : 1); ++h) {
                        if (!wait(&p_ready[h], pp[h], 5u)) break;
                        pp[h] ^= 1u;
                        ptx::tc_fence_after();
                        values(h, vn % NS, st > lo);
                        const bool last = h == 1 || !two;
                        if (last) ptx::mma_commit(&empty[vn % NS]);
                        if (more) {
                            if (h == 0 && !wait(&full[kn % NS], (kn / NS) & 1u, 3u)) break;
                            ptx::tc_fence_after();
                            scores(h, h, kn % NS);
                            ptx::mma_commit(&s_full[h]);
                            if (last) ptx::mma_commit(&empty[kn % NS]);
                        } else {
                            ptx::mma_commit(&o_full[h]);
                        }
                    }
                    if (!ok) break;
                }
            }
            // every product has finished before TMEM is freed
            ptx::mma_commit(&drain_bar);
            const long long t0 = clock64();
            while (!ptx::mbar_try_wait(&drain_bar, 0) && clock64() - t0 < p.wait_limit) {
            }
        }
    } else if (F8 && warp >= 10) {
        // ------------------------------------------------------------ E4M3 codes to fp16
        // a thread has one 16-byte chunk of codes of every KPI-th key (8 or 16: the swizzles stay the same)
        constexpr int CPR = D / 16, KPI = 64 / CPR;
        const int tid = threadIdx.x - 320, key0 = tid / CPR, ch = tid % CPR;
        const int from = key0 * S::ROWB + ((ch ^ (S::ROWB == 128 ? key0 & 7 : (key0 >> 1) & 3)) << 4);
        // its 16 dimensions are two chunks of span ch / 4, which the spans' lanes write in opposite
        // order, for the banks
        const bool swap = (ch >> 2) & 1;
        const int to = (ch >> 2) * S::SPAN + key0 * 128, to_first = ((2 * (ch & 3) + swap) ^ (key0 & 7)) << 4;
        uint32_t n = 0, step_no = 0;
        bool ok = true;
        while (ok && cur.segment(a, G, left, lo, hi)) {
            for (int st = lo; st < hi && ok; ++st, ++step_no) {
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++n) {
                    const uint32_t sl = n % NS, rw = n % NR;
                    ok = ptx::mbar_wait(&raw_full[rw], (n / NR) & 1u, abort_flag, p.wait_limit, a.status, 10u) &&
                         ptx::mbar_wait(&empty[sl], ((n / NS) & 1u) ^ 1u, abort_flag, p.wait_limit, a.status, 11u);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const uint32_t* word = info[step_no % kInfo];
                    const bool partial = (word[0] & word[1] & word[2] & word[3]) != 0xFFFFFFFFu;
                    const unsigned char* src = codes + rw * S::CODES + from;
                    unsigned char* dst = ring + sl * S::SLOT + to;
#pragma unroll 8
                    for (int i = 0; i < TK / KPI; ++i) {
                        uint4 v = *reinterpret_cast<const uint4*>(src + i * KPI * S::ROWB);
                        // keys that are not there count as zero, not as whatever lies there
                        if (partial && !(word[(key0 + i * KPI) >> 5] >> ((key0 + i * KPI) & 31) & 1)) v = make_uint4(0, 0, 0, 0);
                        const uint2 c0 = e4m3x4_to_f16x4(v.x), c1 = e4m3x4_to_f16x4(v.y), c2 = e4m3x4_to_f16x4(v.z), c3 = e4m3x4_to_f16x4(v.w);
                        const uint4 lo16 = make_uint4(c0.x, c0.y, c1.x, c1.y), hi16 = make_uint4(c2.x, c2.y, c3.x, c3.y);
                        *reinterpret_cast<uint4*>(dst + i * KPI * 128 + to_first) = swap ? hi16 : lo16;
                        *reinterpret_cast<uint4*>(dst + i * KPI * 128 + (to_first ^ 16)) = swap ? lo16 : hi16;
                    }
                    ptx::fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        ptx::mbar_arrive(&full[sl]);
                        ptx::mbar_arrive(&raw_free[rw]);
                    }
                }
            }
        }
    } else {
        // ------------------------------------------------------------ softmax of one half
        const int h = warp >> 2, sub = warp & 3;
        const uint32_t s_t = tmem + h * 128 + (static_cast<uint32_t>(sub * 32) << 16);
        const uint32_t o_t = s_t - h * 128 + 256 + h * 128;
        const float all_scale = fmaxf(fabsf(a.scale_log2), 1.0e-37f);   // (0 would turn what is not seen into NaN)
        const uint32_t sign = a.scale_log2 < 0.f ? 0x80008000u : 0u;   // a negative scale: q changes sign instead
        uint32_t sp = 0, op = 0, xp = 0, step_no = 0;
        bool ok = true;
        while (ok && cur.segment(a, G, left, lo, hi)) {
            const SeqInfo s = cur.s;
            const int in_tile = s.n * a.group - cur.mt * G.M;
            const bool share = in_tile <= 128 && hi - lo > 1;          // both halves on the same rows
            const int rows = share ? in_tile : in_tile - h * 128;      // of this half
            if (rows > 0) {
                const int r_first = cur.mt * G.M + (share ? 0 : h * 128);
                // ---- Q to shared memory: a row per D / 8 lanes, 16 bytes each
                // (both halves write the same rows' scales, each its own copy)
                if (!share || h == 0 || F8) {
                    constexpr int LPR = D / 8, RPI = 32 / LPR;
                    unsigned char* dst = smem + h * S::QHALF;
                    const int ch = lane % LPR;                     // 16-byte chunk of the row
                    constexpr int BATCH = 32 / RPI;                // all loads in flight together, before the stores
                    {
                        uint4 in[BATCH];
#pragma unroll
                        for (int k = 0; k < BATCH; ++k) {
                            const int r = sub * 32 + k * RPI + lane / LPR;
                            in[k] = make_uint4(0, 0, 0, 0);
                            if (r < rows) {
                                const int rr = r_first + r, i = token_of(a, rr);
                                in[k] = __ldg(reinterpret_cast<const uint4*>(
                                    a.q + (s.row0 + i) * a.q_stride + static_cast<long long>(cur.h * a.group + rr - i * a.group) * D + ch * 8));
                            }
                        }
#pragma unroll
                        for (int k = 0; k < BATCH; ++k) {
                            const int r = sub * 32 + k * RPI + lane / LPR;
                            uint4 v = make_uint4(in[k].x ^ sign, in[k].y ^ sign, in[k].z ^ sign, in[k].w ^ sign);
                            if constexpr (F8) {
                                // the row's largest finite entry, over the D / 8 lanes that hold it
                                uint32_t w[4] = {v.x, v.y, v.z, v.w};
                                float mx = 0.f;
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const float x = fabsf(__uint_as_float(w[j] << 16)), y = fabsf(__uint_as_float(w[j] & 0xFFFF0000u));
                                    mx = x < INFINITY ? fmaxf(mx, x) : mx;
                                    mx = y < INFINITY ? fmaxf(mx, y) : mx;
                                }
#pragma unroll
                                for (int o = 1; o < LPR; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
                                const int ex = f16_chunk_exp(mx);
                                const float d = exp2_int(-ex);
#pragma unroll
                                for (int j = 0; j < 4; ++j)
                                    w[j] = pack_f16x2(__uint_as_float(w[j] << 16) * d, __uint_as_float(w[j] & 0xFFFF0000u) * d);
                                v = make_uint4(w[0], w[1], w[2], w[3]);
                                if (ch == 0) q_scale[h][r] = all_scale * exp2_int(ex);
                            }
                            *reinterpret_cast<uint4*>(dst + (ch >> 3) * S::SPAN + r * 128 + (((ch & 7) ^ (r & 7)) << 4)) = v;
                        }
                    }
                    ptx::fence_proxy_async_smem();
                    if (!share || h == 0) ptx::mbar_arrive(&q_ready[h]);
                }
                __syncwarp();
                const float scale = F8 ? fmaxf(q_scale[h][sub * 32 + lane], 1.0e-37f) : all_scale;
                const int keys = tile_keys(a, s, cur.mt, G.M);
                const int rr = r_first + min(sub * 32 + lane, rows - 1);   // this thread's row (or the last one)
                const int i = token_of(a, rr);
                // steps that end in front of this key need no look at what a row sees
                const int clear = a.mask != nullptr ? s.ctx : s.ctx + token_of(a, r_first) + 1;
                float m = -INFINITY, l = 0.f;
                const int by = share ? 2 : 1, from = share ? lo + h : lo;
                for (int st = from; st < hi; st += by) {
                    ok = ptx::mbar_wait(&s_full[h], sp, abort_flag, p.wait_limit, a.status, 6u);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    sp ^= 1u;
                    ptx::tc_fence_after();
                    if (sub * 32 >= rows) {                        // no rows here: what lies in P reaches nobody's O
                        ptx::tc_fence_before();
                        ptx::mbar_arrive(&p_ready[h]);
                        continue;
                    }
                    const int c0 = st * TK;
                    const uint32_t* word = info[(step_no + st - lo) % kInfo];
                    const bool masked = c0 + TK > clear || (word[0] & word[1] & word[2] & word[3]) != 0xFFFFFFFFu;
                    uint32_t see[4];
                    if (masked) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) see[q] = seen_bits(a, s, i, c0 + 32 * q, keys) & word[q];
                    }
                    // the maximum over keys 0..63, then over 64..127, which stay in registers
                    uint32_t xa[2][32], xb[2][32];
                    auto hide = [&](uint32_t (&x)[32], int q) {
                        if (masked) {
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(see[q] >> e & 1)) x[e] = 0xFF800000u;
                        }
                    };
                    auto largest = [&](const uint32_t (&x)[32]) {
                        float u = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1])), v = fmaxf(__uint_as_float(x[2]), __uint_as_float(x[3]));
#pragma unroll
                        for (int e = 4; e < 32; e += 4) {
                            u = fmaxf(fmaxf(u, __uint_as_float(x[e])), __uint_as_float(x[e + 1]));
                            v = fmaxf(fmaxf(v, __uint_as_float(x[e + 2])), __uint_as_float(x[e + 3]));
                        }
                        return fmaxf(u, v);
                    };
                    ptx::tmem_ld_32x32b_x32(s_t, xa[0]);
                    ptx::tmem_ld_32x32b_x32(s_t + 32, xa[1]);
                    ptx::tmem_ld_wait(xa[0]);
                    ptx::tmem_ld_wait(xa[1]);
                    hide(xa[0], 0);
                    hide(xa[1], 1);
                    float mx = fmaxf(largest(xa[0]), largest(xa[1]));
                    ptx::tmem_ld_32x32b_x32(s_t + 64, xb[0]);
                    ptx::tmem_ld_32x32b_x32(s_t + 96, xb[1]);
                    ptx::tmem_ld_wait(xb[0]);
                    ptx::tmem_ld_wait(xb[1]);
                    hide(xb[0], 2);
                    hide(xb[1], 3);
                    mx = fmaxf(mx, fmaxf(largest(xb[0]), largest(xb[1])));
                    const bool up = (mx - m) * scale > 8.f || (m == -INFINITY && mx > m);
                    if (__any_sync(0xFFFFFFFFu, up)) {
                        const float m2 = up ? mx : m;
                        const float f = up ? fast_exp2((m - m2) * scale) : 1.f;
                        m = m2;
                        l *= f;
                        if (st > from) {
                            // O so far (complete: its product came before this step's scores)
#pragma unroll
                            for (int q = 0; q < D / 16; ++q) {
                                uint32_t y[16];
                                ptx::tmem_ld_32x32b_x16(o_t + q * 16, y);
                                ptx::tmem_ld_wait16(y);
#pragma unroll
                                for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                                ptx::tmem_st_32x32b_x16(o_t + q * 16, y);
                            }
                        }
                    }
                    const float ref = m == -INFINITY ? 0.f : lifted<F8>(m * scale);
                    const uint64_t scale2 = pair2(scale, scale), ref2 = pair2(-ref, -ref);
                    uint64_t sum2[2] = {0, 0};
                    // P of keys 32 q .. goes where S of later keys was: columns 64 + 16 q ..
                    auto weigh = [&](const uint32_t (&x)[32], int q) {
                        uint32_t pk[16];
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            float u, v;
                            unpair2(fma2(pair2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), scale2, ref2), u, v);
                            u = fast_exp2(u);
                            v = fast_exp2(v);
                            sum2[(e >> 1) & 1] = add2(sum2[(e >> 1) & 1], pair2(u, v));
                            pk[e / 2] = F8 ? pack_f16x2(u, v) : pack_bf16x2(u, v);
                        }
                        ptx::tmem_st_32x32b_x16(s_t + 64 + q * 16, pk);
                    };
                    // keys 0..63 come from TMEM once more, behind the work on the others
                    ptx::tmem_ld_32x32b_x32(s_t, xa[0]);
                    weigh(xb[0], 2);
                    ptx::tmem_ld_32x32b_x32(s_t + 32, xa[1]);
                    weigh(xb[1], 3);
                    ptx::tmem_ld_wait(xa[0]);
                    ptx::tmem_ld_wait(xa[1]);
                    hide(xa[0], 0);
                    hide(xa[1], 1);
                    weigh(xa[0], 0);
                    weigh(xa[1], 1);
                    {
                        float u, v;
                        unpair2(add2(sum2[0], sum2[1]), u, v);
                        l += u + v;
                    }
                    ptx::tmem_st_wait();
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&p_ready[h]);
                }
                step_no += hi - lo;
                if (!ok) break;
                // ---- epilogue: a thread's row of O
                ok = ptx::mbar_wait(&o_full[h], op, abort_flag, p.wait_limit, a.status, 8u);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                op ^= 1u;
                ptx::tc_fence_after();
                float m2 = l == 0.f ? -INFINITY : lifted<F8>(m * scale), f0 = 1.f, f1 = 0.f;
                if (share) {
                    const int x = sub * 32 + lane;
                    if (h == 1) {
                        // the first half reads this half's O; the next one is not begun before it has
                        x_ml[x] = make_float2(m2, l);
                        ptx::tc_fence_before();
                        ptx::mbar_arrive(&x_ready);
                        ok = ptx::mbar_wait(&x_done, xp, abort_flag, p.wait_limit, a.status, 12u);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        xp ^= 1u;
                        continue;
                    }
                    ok = ptx::mbar_wait(&x_ready, xp, abort_flag, p.wait_limit, a.status, 13u);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    xp ^= 1u;
                    ptx::tc_fence_after();
                    const float2 o = x_ml[x];
                    const float both = fmaxf(m2, o.x), base = both == -INFINITY ? 0.f : both;
                    f0 = fast_exp2(m2 - base);
                    f1 = fast_exp2(o.x - base);
                    m2 = both;
                    l = l * f0 + o.y * f1;
                }
                const bool mine = sub * 32 + lane < rows;
                const int head = cur.h * a.group + rr - i * a.group;
                const long long row = s.row0 + i;
                const bool whole = lo == 0 && hi == cur.steps;
                const size_t slot_row = (2 * static_cast<size_t>(blockIdx.x) + (lo == 0)) * kTileRows + h * 128 + sub * 32 + lane;   // (share: h is 0)
                if (threadIdx.x == 0 && lo == 0 && !whole)         // (the last of the share; half 0 always has rows)
                    p.part.items[blockIdx.x] =
                        JoinItem{item_shares(shares, cur, G, x1, left).y, s.row0, s.n * a.group, cur.h, cur.mt};
                float* part_o = p.part.o + slot_row * D;
                float* part_ml = p.part.ml + slot_row * 2;
                const float inv = l == 0.f ? 0.f : __fdividef(a.c.v_scale, l);
                // a row of O, 32 dimensions at a time, and whether it holds NaN
                auto take = [&](int q, uint32_t (&x)[32]) {
                    ptx::tmem_ld_32x32b_x32(o_t + q * 32, x);
                    ptx::tmem_ld_wait(x);
                    if (share) {
                        uint32_t y[32];
                        ptx::tmem_ld_32x32b_x32(o_t + 128 + q * 32, y);
                        ptx::tmem_ld_wait(y);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            x[e] = __float_as_uint(__uint_as_float(x[e]) * f0 + __uint_as_float(y[e]) * f1);
                    }
                    bool n = false;
#pragma unroll
                    for (int e = 0; e < 32; ++e) n |= __uint_as_float(x[e]) != __uint_as_float(x[e]);
                    return n;
                };
                const bool unseen = hi * TK > s.ctx;               // the item has keys that some row may not see
                bool nan = false, stays = false;
                if (unseen && whole && a.out == a.q) {
                    // in place: a row that is computed again below still needs its query
#pragma unroll 1
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t x[32];
                        stays |= take(q, x);
                    }
                    const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, mine && stays && l == l);
                    stays = lanes != 0 && (spoiled_lanes<D, F8>(a, cur, i, lanes, lo * TK, min(hi * TK, keys), lane) >> lane & 1);
                }
#pragma unroll
                for (int q = 0; q < D / 32; ++q) {
                    uint32_t x[32];
                    nan |= take(q, x);
                    if (mine && whole && !stays) {
                        uint4* dst = reinterpret_cast<uint4*>(a.out + row * a.out_stride + head * D + q * 32);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t w[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                w[j] = l == 0.f ? 0u : pack_bf16x2(__uint_as_float(x[e * 8 + 2 * j]) * inv,
                                                                   __uint_as_float(x[e * 8 + 2 * j + 1]) * inv);
                            dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    } else if (mine && !whole) {
                        uint4* dst = reinterpret_cast<uint4*>(part_o + q * 32);
#pragma unroll
                        for (int e = 0; e < 8; ++e) dst[e] = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
                    }
                    __syncwarp();
                }
                ptx::tc_fence_before();
                if (share) ptx::mbar_arrive(&x_done);
                if (mine) {
                    if (!whole) {
                        part_ml[0] = m2;
                        part_ml[1] = l;
                    } else if (a.lse != nullptr) {
                        a.lse[row * a.n_q + head] = lse_of(m2, l);
                    }
                }
                // 0 * infinity or NaN: a value that the row may not see; again, key by key
                __syncwarp();
                const uint32_t again = __ballot_sync(0xFFFFFFFFu, mine && nan && l == l && unseen);
                if (again)
                    redo_rows<D, F8>(a, cur, again, i, head, lo * TK, min(hi * TK, keys), whole ? nullptr : p.part.o + (slot_row - lane) * D,
                                     p.part.ml + (slot_row - lane) * 2, lane);
            } else {
                step_no += hi - lo;
            }
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <int D, bool F8>
cudaError_t launch_tiles(const AttnArgs& a, void* partials, int sms, cudaStream_t st) {
    using S = Tile<D, F8>;
    TileParams p;
    p.a = a;
    const int page = 1 << a.c.page_shift;
    const int box = page < TK ? page : TK;
    p.box_shift = page < TK ? a.c.page_shift : 7;
    p.stall = tree_attn_take_stall();
    p.wait_limit = p.stall ? 20ll << 20 : tile_wait_limit(a);
    if (!make_kv_map(&p.tk, a, false, box) || !make_kv_map(&p.tv, a, true, box)) return cudaErrorInvalidValue;
    const int blocks = sms < kTileBlocks ? sms : kTileBlocks;
    p.part = partials_at(partials, blocks, kTileRows);
    const cudaError_t e = cudaFuncSetAttribute(tiles_kernel<D, F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    {
        ProfileScope ps("tree_attention", st);
        tiles_kernel<D, F8><<<blocks, F8 ? TL_THREADS_F8 : TL_THREADS, S::SMEM, st>>>(p);
        note_launch();
    }
    const cudaError_t le = cudaGetLastError();
    if (le != cudaSuccess) return le;
    return launch_tree_attn_join(a, kTileRows, p.part, blocks, st);
}

}  // namespace

bool tree_attn_tiles_apply(const AttnArgs& a) {
    return a.head_dim <= 128 && static_cast<long long>(a.c.max_new) * a.group > kTileLeastRows && !tree_attn_short(a);
}

cudaError_t launch_tree_attn_tiles(const AttnArgs& a, void* partials, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (sms <= 0) sms = 148;
    if (a.head_dim == 64) return a.f8 ? launch_tiles<64, true>(a, partials, sms, st) : launch_tiles<64, false>(a, partials, sms, st);
    return a.f8 ? launch_tiles<128, true>(a, partials, sms, st) : launch_tiles<128, false>(a, partials, sms, st);
}

}  // namespace sre
