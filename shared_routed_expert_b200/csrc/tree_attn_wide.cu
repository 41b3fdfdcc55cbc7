// Attention over a paged cache for many query rows per kv head and heads of 256 dimensions: the
// products of tree_attn_tiles.cu with one tile of 128 packed query rows per block, since O alone
// takes half of TMEM:
//   S_b = Q K^T          two S of 128 keys in turn (b), so that the next step's scores are formed
//                        while this step's exponentials run
//   P_b = 2^(S_b - m)    four warps, one thread per row; P overwrites S in TMEM
//   O  += P_b V          256 columns of TMEM
// K and V come as halves of 128 dimensions (32 KB of 16-bit values each), so the ring in shared
// memory keeps the slots of the narrower kernel beside 64 KB of Q. Each half is freed when its
// product has read it. The maximum is raised only when a row's grows by more than 2^8; O is
// rescaled after the product in front has finished. 128 exponentials per thread and step stand
// against four products of 128 x 128 x 128, as there; with 192 threads a row of S stays in registers.
// Measured, 16 heads over 4 kv heads, bf16: 4096 rows behind 4096 keys 408 us, 1010 TFLOP/s (the 16-row
// products of tree_attn_small.cu: 1944 us), 1024 rows behind 2048 keys 75 us; E4M3 108 to 120 us, bound
// by the conversion (two warps instead of four: 130 us).
// Roles: warps 0-3 softmax, loads of Q and epilogue; warp 4 the products; warp 5 streams K and V;
// E4M3: warps 6 to 9 convert codes to fp16. Every wait is bounded.
#include "kernels.cuh"
#include "tc_ptx.cuh"
#include "tree_attn.cuh"

namespace sre {

namespace {

constexpr int TK = 128;                  // keys per step
constexpr int WD_THREADS = 192, WD_CONVERT = 4, WD_THREADS_F8 = WD_THREADS + 32 * WD_CONVERT;
constexpr int kWideExtra = 4;            // what an item costs besides its steps, in steps
// Rows of a kv head from which this kernel takes over: 32 sequences of 9 rows of 16 heads (36 rows a
// kv head), 568 MB of bf16 cache 105 us here, 183 us there, E4M3 147 and 202 us; of 7 rows (28), two
// passes there, 109 and 116 us there.
constexpr int kWideLeastRows = 32;
constexpr int kWideLeastShare = 3;       // units of the shortest share
constexpr int kInfo = 8;                 // steps whose key masks are kept (the producer is at most 4 ahead)

template <bool F8>
struct Wide {
    static constexpr int D = 256;
    static constexpr int SPAN = 128 * 128;                         // bytes of a span (128 bytes of each of 128 rows)
    static constexpr int QBYTES = D * 2 / 128 * SPAN;
    static constexpr int SLOT = 2 * SPAN;                          // 128 dimensions of a step's K or V, 16 bits each
    static constexpr int NS = F8 ? 3 : 5;
    static constexpr int NR = F8 ? 4 : 0;                          // as codes: one span
    static constexpr int SMEM = QBYTES + NS * SLOT + NR * SPAN + 1024;
    static constexpr int LOAD_SPANS = F8 ? 1 : 2;                  // spans of a half, as they are loaded
};

struct WideParams {
    AttnArgs a;
    CUtensorMap tk, tv;
    Partials part;
    int box_shift;
    long long wait_limit;
    bool stall;                          // testing: no loads
};

template <bool F8>
__global__ void __launch_bounds__(F8 ? WD_THREADS_F8 : WD_THREADS, 1) wide_kernel(const __grid_constant__ WideParams p) {
    using S = Wide<F8>;
    constexpr int D = S::D, NS = S::NS, NR = S::NR > 0 ? S::NR : 1;
    constexpr Tiling G{kWideRows, TK, kWideExtra};
    extern __shared__ __align__(1024) unsigned char wd_raw[];
    __shared__ ScanShared scan;
    __shared__ uint64_t full[NS], empty[NS], q_ready, s_full[2], p_ready[2], o_done[2], tail_bar, drain_bar;
    __shared__ uint64_t raw_full[NR], raw_free[NR];
    __shared__ uint32_t info[kInfo][4];  // keys of a step that were loaded
    __shared__ uint32_t tmem_base_s;
    __shared__ int s_abort;
    unsigned char* smem = wd_raw + ((1024 - (ptx::smem_u32(wd_raw) & 1023)) & 1023);
    unsigned char* ring = smem + S::QBYTES;
    unsigned char* codes = ring + NS * S::SLOT;
    volatile int* abort_flag = &s_abort;
    const AttnArgs& a = p.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int i = 0; i < NS; ++i) {
            ptx::mbar_init(&full[i], F8 ? WD_CONVERT : 1);
            ptx::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NR; ++i) {
            ptx::mbar_init(&raw_full[i], 1);
            ptx::mbar_init(&raw_free[i], WD_CONVERT);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&s_full[i], 1);
            ptx::mbar_init(&p_ready[i], 128);
            ptx::mbar_init(&o_done[i], 1);
        }
        ptx::mbar_init(&q_ready, 128);
        ptx::mbar_init(&tail_bar, 1);
        ptx::mbar_init(&drain_bar, 1);
        ptx::fence_mbar_init();
        ptx::prefetch_tmap(&p.tk);
        ptx::prefetch_tmap(&p.tv);
    }
    ScanThread me;
    const long long W = scan_units(a, G, scan, me);
    const Shares shares(W, gridDim.x, kWideLeastShare);
    if (threadIdx.x == 0) p.part.items[blockIdx.x].parts = 0;
    if (static_cast<int>(blockIdx.x) >= shares.count) return;
    const long long x0 = shares.begin(blockIdx.x), x1 = shares.begin(blockIdx.x + 1);
    Cursor cur = seek(a, G, scan, x0, me);
    long long left = x1 - x0;
    int lo, hi;
    if (warp == 4) {
        ptx::tmem_alloc(&tmem_base_s, 512);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = tmem_base_s;   // columns: S0 0, S1 128, O 256

    // The halves of K and V of an item lie in the ring in the order the products take them:
    // K of the first step, then for each step K of the next one and V of its own.
    if (warp == 5) {
        // ------------------------------------------------------------ producer
        const int box = 1 << p.box_shift, pieces = TK >> p.box_shift;
        uint32_t n = 0, step_no = 0, tail_phase = 0;               // slots and steps so far
        bool ok = !p.stall;
        // a step's pieces: lane q < pieces has piece q
        struct Step {
            int page, slot;
            bool good, partial;
            uint32_t goods, word;                                  // word: lane q < 4, keys 32 q .. that are there
        };
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
            auto look = [&](int st) {
                Step x;
                const int c0 = st * TK;
                const int at = (c0 - first) >> p.box_shift;
                if (at - base >= 32) {                             // (pieces per step divide 32)
                    base += 32;
                    page_now = page_next;
                    page_next = fetch(base + 32);
                }
                x.page = __shfl_sync(0xFFFFFFFFu, page_now, (at - base + lane) & 31);
                const int c = c0 + (lane << p.box_shift);
                const bool wanted = lane < pieces && c < keys;
                x.good = wanted && x.page >= 0 && x.page < a.c.num_pages;
                if (wanted && !x.good) report(a.status, MOE_ERR_DEVICE, cur.b);
                x.goods = __ballot_sync(0xFFFFFFFFu, x.good);
                x.word = 0xFFFFFFFFu;
                const int k0 = lane * 32, rest = keys - (c0 + k0);
                if (rest < 32) x.word = rest <= 0 ? 0u : (1u << rest) - 1u;
                if (box >= 32) {
                    if (!(x.goods >> ((k0 >> p.box_shift) & 31) & 1)) x.word = 0;
                } else {
                    if (!(x.goods >> ((2 * lane) & 31) & 1)) x.word &= 0xFFFF0000u;
                    if (!(x.goods >> ((2 * lane + 1) & 31) & 1)) x.word &= 0xFFFFu;
                }
                if (lane < 4) info[(step_no + st - lo) % kInfo][lane] = x.word;
                __syncwarp();
                x.partial = __any_sync(0xFFFFFFFFu, lane < 4 && x.word != 0xFFFFFFFFu);
                x.slot = c & ((1 << a.c.page_shift) - 1);
                return x;
            };
            auto load = [&](const Step& x, bool is_v) {
                const uint32_t bytes = static_cast<uint32_t>(__popc(x.goods)) * box * 128 * S::LOAD_SPANS;
#pragma unroll 1
                for (int half = 0; half < 2; ++half, ++n) {
                    const uint32_t sl = F8 ? n % NR : n % NS, use = F8 ? n / NR : n / NS;
                    ok = ok && ptx::mbar_wait(F8 ? &raw_free[sl] : &empty[sl], (use & 1u) ^ 1u, abort_flag, p.wait_limit, a.status, 1u);
                    ok = __all_sync(0xFFFFFFFFu, ok);
                    if (!ok) break;
                    const bool tail = !F8 && is_v && x.partial;
                    uint64_t* bar = F8 ? &raw_full[sl] : (tail ? &tail_bar : &full[sl]);
                    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, bytes);
                    __syncwarp();
                    unsigned char* dst = F8 ? codes + sl * S::SPAN : ring + sl * S::SLOT;
                    if (x.good) {
#pragma unroll
                        for (int sp = 0; sp < S::LOAD_SPANS; ++sp)
                            ptx::tma_load_5d(dst + sp * S::SPAN + lane * box * 128, is_v ? &p.tv : &p.tk, bar, 0, x.slot,
                                             half * S::LOAD_SPANS + sp, cur.h, x.page);
                    }
                    if (tail) {
                        // keys that are not there count as zero, not as 0 * whatever lies there
                        ok = ptx::mbar_wait(&tail_bar, tail_phase, abort_flag, p.wait_limit, a.status, 7u);
                        tail_phase ^= 1u;
                        ok = __all_sync(0xFFFFFFFFu, ok);
#pragma unroll 1
                        for (int r = lane; r < TK; r += 32) {
                            const uint32_t w = __shfl_sync(0xFFFFFFFFu, x.word, r >> 5);
                            if (w >> (r & 31) & 1) continue;
                            for (int sp = 0; sp < 2; ++sp)
#pragma unroll
                                for (int ch = 0; ch < 8; ++ch)
                                    *reinterpret_cast<uint4*>(dst + sp * S::SPAN + r * 128 + ch * 16) = make_uint4(0, 0, 0, 0);
                        }
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(&full[sl]);
                    }
                }
            };
            Step now = look(lo);
            load(now, false);
            for (int st = lo; st < hi && ok; ++st) {
                Step next = now;
                if (st + 1 < hi) {
                    next = look(st + 1);
                    load(next, false);
                }
                if (ok) load(now, true);
                now = next;
            }
            step_no += hi - lo;
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
    } else if (warp == 4) {
        // ------------------------------------------------------------ products
        if (lane == 0) {
            constexpr uint32_t IS = ptx::instr_desc(128, TK, F8 ? 0 : 1);
            constexpr uint32_t IO = ptx::instr_desc(128, 128, F8 ? 0 : 1) | ptx::kBMnMajor;
            const uint32_t q_u = ptx::smem_u32(smem), ring_u = ptx::smem_u32(ring);
            uint32_t n = 0, steps = 0, qp = 0;
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
            auto scores = [&](uint32_t b) {
#pragma unroll 1
                for (int half = 0; half < 2; ++half, ++n) {
                    if (!wait(&full[n % NS], (n / NS) & 1u, 3u)) return;
                    ptx::tc_fence_after();
                    const uint32_t ka = k_lo + ((ring_u + (n % NS) * S::SLOT) >> 4), qa = k_lo + ((q_u + half * S::SLOT) >> 4);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t off = ((k >> 2) * S::SPAN + (k & 3) * 32) >> 4;
                        ptx::mma_f16(tmem + b * 128, desc(k_hi, qa + off), desc(k_hi, ka + off), IS, half != 0 || k != 0);
                    }
                    ptx::mma_commit(&empty[n % NS]);
                }
                ptx::mma_commit(&s_full[b]);
            };
            while (ok && cur.segment(a, G, left, lo, hi)) {
                if (!wait(&q_ready, qp, 4u)) break;
                qp ^= 1u;
                scores(steps & 1u);
                for (int st = lo; st < hi && ok; ++st, ++steps) {
                    const uint32_t b = steps & 1u;
                    // (the other S has been read: its P was waited for, and its product came first)
                    if (st + 1 < hi) scores(b ^ 1u);
                    if (!ok || !wait(&p_ready[b], (steps >> 1) & 1u, 5u)) break;
#pragma unroll 1
                    for (int half = 0; half < 2; ++half, ++n) {
                        if (!wait(&full[n % NS], (n / NS) & 1u, 9u)) break;
                        ptx::tc_fence_after();
                        const uint32_t va = mn_lo + ((ring_u + (n % NS) * S::SLOT) >> 4);
#pragma unroll
                        for (int k = 0; k < TK / 16; ++k)
                            ptx::mma_f16_ts(tmem + 256 + half * 128, tmem + b * 128 + 64 + k * 8, desc(mn_hi, va + k * 128), IO,
                                            st > lo || k != 0);
                        ptx::mma_commit(&empty[n % NS]);
                    }
                    if (!ok) break;
                    ptx::mma_commit(&o_done[b]);
                }
            }
            // every product has finished before TMEM is freed
            ptx::mma_commit(&drain_bar);
            const long long t0 = clock64();
            while (!ptx::mbar_try_wait(&drain_bar, 0) && clock64() - t0 < p.wait_limit) {
            }
        }
    } else if (F8 && warp >= 6) {
        // ------------------------------------------------------------ E4M3 codes to fp16
        // (as in tree_attn_tiles.cu: a thread has one 16-byte chunk of codes of every KPI-th key)
        constexpr int KPI = 4 * WD_CONVERT;                        // (a multiple of 8: the swizzles stay the same)
        const int tid = threadIdx.x - 192, key0 = tid >> 3, ch = tid & 7;
        const int from = key0 * 128 + ((ch ^ (key0 & 7)) << 4);
        const bool swap = (ch >> 2) & 1;
        const int to = (ch >> 2) * S::SPAN + key0 * 128, to_first = ((2 * (ch & 3) + swap) ^ (key0 & 7)) << 4;
        uint32_t n = 0, step_no = 0;
        bool ok = true;
        auto convert = [&](uint32_t step) {
#pragma unroll 1
            for (int half = 0; half < 2 && ok; ++half, ++n) {
                const uint32_t sl = n % NS, rw = n % NR;
                ok = ptx::mbar_wait(&raw_full[rw], (n / NR) & 1u, abort_flag, p.wait_limit, a.status, 10u) &&
                     ptx::mbar_wait(&empty[sl], ((n / NS) & 1u) ^ 1u, abort_flag, p.wait_limit, a.status, 11u);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const uint32_t* word = info[step % kInfo];
                const bool partial = (word[0] & word[1] & word[2] & word[3]) != 0xFFFFFFFFu;
                const unsigned char* src = codes + rw * S::SPAN + from;
                unsigned char* dst = ring + sl * S::SLOT + to;
#pragma unroll 8
                for (int i = 0; i < TK / KPI; ++i) {
                    uint4 v = *reinterpret_cast<const uint4*>(src + i * KPI * 128);
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
        };
        while (ok && cur.segment(a, G, left, lo, hi)) {
            convert(step_no);
            for (int st = lo; st < hi && ok; ++st, ++step_no) {
                if (st + 1 < hi) convert(step_no + 1);
                if (ok) convert(step_no);
            }
        }
    } else {
        // ------------------------------------------------------------ softmax, Q, epilogue
        const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
        const uint32_t o_t = tmem + 256 + lanes;
        const float all_scale = fmaxf(fabsf(a.scale_log2), 1.0e-37f);   // (0 would turn what is not seen into NaN)
        const uint32_t sign = a.scale_log2 < 0.f ? 0x80008000u : 0u;   // a negative scale: q changes sign instead
        uint32_t steps = 0;
        bool ok = true;
        while (ok && cur.segment(a, G, left, lo, hi)) {
            const SeqInfo s = cur.s;
            const int rows = s.n * a.group - cur.mt * G.M;
            const int r_first = cur.mt * G.M;
            float scale = all_scale;
            // ---- Q to shared memory: a row per instruction, 16 bytes a lane, 16 rows in flight
#pragma unroll 1
            for (int r0 = warp * 32; r0 < warp * 32 + 32; r0 += 16) {
                uint4 in[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    in[k] = make_uint4(0, 0, 0, 0);
                    if (r0 + k < rows) {
                        const int rr = r_first + r0 + k, i = token_of(a, rr);
                        in[k] = __ldg(reinterpret_cast<const uint4*>(
                            a.q + (s.row0 + i) * a.q_stride + static_cast<long long>(cur.h * a.group + rr - i * a.group) * D + lane * 8));
                    }
                }
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const int r = r0 + k;
                    uint4 v = make_uint4(in[k].x ^ sign, in[k].y ^ sign, in[k].z ^ sign, in[k].w ^ sign);
                    if constexpr (F8) {
                        // the row's largest finite entry
                        uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        float mx = 0.f;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float x = fabsf(__uint_as_float(w[j] << 16)), y = fabsf(__uint_as_float(w[j] & 0xFFFF0000u));
                            mx = x < INFINITY ? fmaxf(mx, x) : mx;
                            mx = y < INFINITY ? fmaxf(mx, y) : mx;
                        }
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
                        const int ex = f16_chunk_exp(mx);
                        const float d = exp2_int(-ex);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = pack_f16x2(__uint_as_float(w[j] << 16) * d, __uint_as_float(w[j] & 0xFFFF0000u) * d);
                        v = make_uint4(w[0], w[1], w[2], w[3]);
                        if (lane == (r & 31)) scale = fmaxf(all_scale * exp2_int(ex), 1.0e-37f);
                    }
                    *reinterpret_cast<uint4*>(smem + (lane >> 3) * S::SPAN + r * 128 + (((lane & 7) ^ (r & 7)) << 4)) = v;
                }
            }
            ptx::fence_proxy_async_smem();
            ptx::mbar_arrive(&q_ready);
            const int keys = tile_keys(a, s, cur.mt, G.M);
            const int rr = r_first + min(warp * 32 + lane, rows - 1);      // this thread's row (or the last one)
            const int i = token_of(a, rr);
            // steps that end in front of this key need no look at what a row sees
            const int clear = a.mask != nullptr ? s.ctx : s.ctx + token_of(a, r_first) + 1;
            float m = -INFINITY, l = 0.f;
            for (int st = lo; st < hi; ++st, ++steps) {
                const uint32_t b = steps & 1u, s_t = tmem + b * 128 + lanes;
                ok = ptx::mbar_wait(&s_full[b], (steps >> 1) & 1u, abort_flag, p.wait_limit, a.status, 6u);
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                ptx::tc_fence_after();
                if (warp * 32 >= rows) {                           // no rows here: what lies in P reaches nobody's O
                    ptx::tc_fence_before();
                    ptx::mbar_arrive(&p_ready[b]);
                    continue;
                }
                const int c0 = st * TK;
                const uint32_t* word = info[steps % kInfo];
                const bool masked = c0 + TK > clear || (word[0] & word[1] & word[2] & word[3]) != 0xFFFFFFFFu;
                uint32_t x[4][32];
#pragma unroll
                for (int q = 0; q < 4; ++q) ptx::tmem_ld_32x32b_x32(s_t + 32 * q, x[q]);
#pragma unroll
                for (int q = 0; q < 4; ++q) ptx::tmem_ld_wait(x[q]);
                if (masked) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t see = seen_bits(a, s, i, c0 + 32 * q, keys) & word[q];
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!(see >> e & 1)) x[q][e] = 0xFF800000u;
                    }
                }
                float u = -INFINITY, v = -INFINITY;
#pragma unroll
                for (int q = 0; q < 4; ++q)
#pragma unroll
                    for (int e = 0; e < 32; e += 4) {
                        u = fmaxf(fmaxf(u, __uint_as_float(x[q][e])), __uint_as_float(x[q][e + 1]));
                        v = fmaxf(fmaxf(v, __uint_as_float(x[q][e + 2])), __uint_as_float(x[q][e + 3]));
                    }
                const float mx = fmaxf(u, v);
                const bool up = (mx - m) * scale > 8.f || (m == -INFINITY && mx > m);
                if (__any_sync(0xFFFFFFFFu, up)) {
                    const float m2 = up ? mx : m;
                    const float f = up ? fast_exp2((m - m2) * scale) : 1.f;
                    m = m2;
                    l *= f;
                    if (st > lo) {
                        // O so far, when the product in front has finished
                        ok = ptx::mbar_wait(&o_done[(steps - 1) & 1u], ((steps - 1) >> 1) & 1u, abort_flag, p.wait_limit, a.status, 12u);
                        ok = __all_sync(0xFFFFFFFFu, ok);
                        if (!ok) break;
                        ptx::tc_fence_after();
#pragma unroll 1
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
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float g0, g1;
                        unpair2(fma2(pair2(__uint_as_float(x[q][e]), __uint_as_float(x[q][e + 1])), scale2, ref2), g0, g1);
                        g0 = fast_exp2(g0);
                        g1 = fast_exp2(g1);
                        sum2[(e >> 1) & 1] = add2(sum2[(e >> 1) & 1], pair2(g0, g1));
                        pk[e / 2] = F8 ? pack_f16x2(g0, g1) : pack_bf16x2(g0, g1);
                    }
                    ptx::tmem_st_32x32b_x16(s_t + 64 + q * 16, pk);
                }
                unpair2(add2(sum2[0], sum2[1]), u, v);
                l += u + v;
                ptx::tmem_st_wait();
                ptx::tc_fence_before();
                ptx::mbar_arrive(&p_ready[b]);
            }
            if (!ok) break;
            // ---- epilogue: a thread's row of O
            ok = ptx::mbar_wait(&o_done[(steps - 1) & 1u], ((steps - 1) >> 1) & 1u, abort_flag, p.wait_limit, a.status, 8u);
            ok = __all_sync(0xFFFFFFFFu, ok);
            if (!ok) break;
            ptx::tc_fence_after();
            const float m2 = l == 0.f ? -INFINITY : lifted<F8>(m * scale);
            const bool mine = warp * 32 + lane < rows;
            const int head = cur.h * a.group + rr - i * a.group;
            const long long row = s.row0 + i;
            const bool whole = lo == 0 && hi == cur.steps;
            const size_t slot_row = (2 * static_cast<size_t>(blockIdx.x) + (lo == 0)) * kWideRows + warp * 32 + lane;
            if (threadIdx.x == 0 && lo == 0 && !whole)             // (the last of the share)
                p.part.items[blockIdx.x] = JoinItem{item_shares(shares, cur, G, x1, left).y, s.row0, s.n * a.group, cur.h, cur.mt};
            float* part_o = p.part.o + slot_row * D;
            const float inv = l == 0.f ? 0.f : __fdividef(a.c.v_scale, l);
            auto take = [&](int q, uint32_t (&x)[32]) {            // 32 dimensions of the row, and whether they hold NaN
                ptx::tmem_ld_32x32b_x32(o_t + q * 32, x);
                ptx::tmem_ld_wait(x);
                bool n = false;
#pragma unroll
                for (int e = 0; e < 32; ++e) n |= __uint_as_float(x[e]) != __uint_as_float(x[e]);
                return n;
            };
            const bool unseen = hi * TK > s.ctx;                   // the item has keys that some row may not see
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
#pragma unroll 1
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
            if (mine) {
                if (!whole) *reinterpret_cast<float2*>(p.part.ml + slot_row * 2) = make_float2(m2, l);
                else if (a.lse != nullptr) a.lse[row * a.n_q + head] = lse_of(m2, l);
            }
            // 0 * infinity or NaN: a value that the row may not see; again, key by key
            __syncwarp();
            const uint32_t again = __ballot_sync(0xFFFFFFFFu, mine && nan && l == l && unseen);
            if (again)
                redo_rows<D, F8>(a, cur, again, i, head, lo * TK, min(hi * TK, keys), whole ? nullptr : p.part.o + (slot_row - lane) * D,
                                 p.part.ml + (slot_row - lane) * 2, lane);
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 4) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <bool F8>
cudaError_t launch_wide(const AttnArgs& a, void* partials, int sms, cudaStream_t st) {
    using S = Wide<F8>;
    WideParams p;
    p.a = a;
    const int page = 1 << a.c.page_shift;
    const int box = page < TK ? page : TK;
    p.box_shift = page < TK ? a.c.page_shift : 7;
    p.stall = tree_attn_take_stall();
    p.wait_limit = p.stall ? 20ll << 20 : tile_wait_limit(a);
    if (!make_kv_map(&p.tk, a, false, box) || !make_kv_map(&p.tv, a, true, box)) return cudaErrorInvalidValue;
    const int blocks = sms < kTileBlocks ? sms : kTileBlocks;
    p.part = partials_at(partials, blocks, kWideRows);
    const cudaError_t e = cudaFuncSetAttribute(wide_kernel<F8>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    {
        ProfileScope ps("tree_attention", st);
        wide_kernel<F8><<<blocks, F8 ? WD_THREADS_F8 : WD_THREADS, S::SMEM, st>>>(p);
        note_launch();
    }
    const cudaError_t le = cudaGetLastError();
    if (le != cudaSuccess) return le;
    return launch_tree_attn_join(a, kWideRows, p.part, blocks, st);
}

}  // namespace

bool tree_attn_wide_apply(const AttnArgs& a) {
    return a.head_dim == 256 && static_cast<long long>(a.c.max_new) * a.group > kWideLeastRows && !tree_attn_short(a);
}

cudaError_t launch_tree_attn_wide(const AttnArgs& a, void* partials, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (sms <= 0) sms = 148;
    return a.f8 ? launch_wide<true>(a, partials, sms, st) : launch_wide<false>(a, partials, sms, st);
}

}  // namespace sre
