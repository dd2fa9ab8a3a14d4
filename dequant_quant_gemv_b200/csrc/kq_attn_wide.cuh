// kq_attn_wide.cuh — attention where a pair has many query rows (verify of
// several columns of many heads): up to 128 rows, tcgen05.
//
// The block is one stream.  The rows of a pair are the M of both products:
// scores (128 x 64 keys) and weighted values (128 x D) come out of tcgen05.mma
// into tensor memory, a thread per row reads them back, and keys and values are
// read from HBM and shared memory once for all rows.  The queries' and the
// weights' 16-bit terms are operands in tensor memory, too: from shared memory
// a product of 128 x 64 x 16 takes 48 cycles, from there 31.  The sums over the
// chunks are in registers, so that every chunk starts from zero, as in the
// kernel for few rows.
//
// Roles: four warps of softmax; four that sum the weighted values; one that
// issues the products; one that copies keys and one that copies values, three
// chunks on their way.  They hand each other chunks through barriers in shared
// memory, every wait bounded: one that runs out sets the fault word and ends the
// block's roles, and what is in flight lands before the block exits.  The products of a chunk wait on one barrier, at
// which the softmax (4 warps), the sums of the chunk before (4) and the values (1)
// arrive.  While the softmax of a chunk runs, the weighted values of the chunk
// before are made, and the scores of the next.
//
// Measured (device time): 4 requests of 3001 to 16000 keys, verify of 8 columns, 64
// rows per pair, bf16: 70 us for 138 MB (107 with tiles of 16 rows); 4 of 4000
// keys, 128 rows, bf16: 52 us (109).  A chunk takes about 3000 cycles, bound by
// the chain softmax (1000), weights' terms (900), values' products (1100) and
// the waits between; the scores' products (900) and the sums (600) run beside
// it.
#pragma once

#include "kq_attn.cuh"

namespace kq {

constexpr int kWideChunk = 64;

// Shared-memory matrix descriptors (128-byte swizzle; atoms of 8 rows of 128
// bytes): rows along M or N with K contiguous, and, for the values, K along
// the rows with N contiguous (blocks of 64 dimensions `lbo` bytes apart).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo) {
    return static_cast<uint64_t>((addr & 0x3ffffu) >> 4) | static_cast<uint64_t>(lbo >> 4) << 16 |
           static_cast<uint64_t>(1024 >> 4) << 32 | 1ull << 46 | 2ull << 61;
}

// The lane that issues (under a branch on lane == 0 a product of 64 keys takes 49
// cycles, under this one 32).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// One thread's product of 128 x N x 16.  A is in tensor memory, two values of K per column.
__device__ __forceinline__ void mma_tc(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
}

// 16 columns of the warp's 32 lanes of tensor memory.
__device__ __forceinline__ void tmem_store16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// 32 consecutive columns of the warp's 32 lanes of tensor memory.
__device__ __forceinline__ void tmem_load32(float (&v)[32], uint32_t addr) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Chunks in the ring: what shared memory holds beside the rest, four at most.
template <int D>
constexpr int kWideStages = D == 128 ? 3 : 4;

// Alignment, the weights of a chunk whose values are not all finite, queries on
// their way, the ring.
template <int D>
constexpr int kWideSmem = 1024 + 128 * kWideChunk * 4 + 128 * D * 4 + kWideStages<D> * 2 * (D / 64) * 8192;

// `bytes` (4 or 8) from global to shared memory, zeros when !in.
template <int BYTES>
__device__ __forceinline__ void copy_small(uint32_t to, const void* from, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(BYTES), "r"(in ? BYTES : 0)
                 : "memory");
}

constexpr int kWideThreads = 32 * (kAttnWarps + 4);

template <int D, bool BF16>
__global__ void __launch_bounds__(kWideThreads, 1) attn_wide_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int TERMS = BF16 ? 3 : 2, TR = 16, PF = kPart<D, TR>;
    constexpr int CK = kWideChunk, DB = D / 64;           // blocks of 64 dimensions
    constexpr uint32_t HALF = DB * 8192;                  // bytes of a chunk's keys, or values
    // tensor memory: weighted values, two chunks' scores and weights, queries.
    // Three terms of 128 dimensions leave no room for both of the former: the weights
    // come to the scores' columns, and the next scores wait until they were used.
    constexpr uint32_t kCols = 512, QT = D / 2, PT = CK / 2;
    constexpr bool OVER = D + 2 * CK + TERMS * (2 * PT + QT) > kCols;
    constexpr uint32_t kColS = D, kBuf = OVER ? TERMS * PT : CK;
    constexpr uint32_t kColP = OVER ? kColS : kColS + 2 * CK, kColQ = kColP + 2 * TERMS * PT;
    static_assert(kBuf >= CK && kColQ + TERMS * QT <= kCols, "tensor memory");
    constexpr int STG = kWideStages<D>;
    constexpr int TGT = BF16 ? 0 : 14;
    constexpr uint32_t TYPE = BF16 ? 1u : 0u;
    constexpr uint32_t IDESC = 1u << 4 | TYPE << 7 | TYPE << 10 | (128u >> 4) << 24;
    constexpr uint32_t IDESC_S = IDESC | (static_cast<uint32_t>(CK) >> 3) << 17;
    constexpr uint32_t IDESC_Y = IDESC | 1u << 16 | (static_cast<uint32_t>(D) >> 3) << 17;

    extern __shared__ __align__(1024) uint8_t wide_smem[];
    __shared__ int sums[kAttnWarps * 32], wsum[kAttnWarps];
    __shared__ int3 kept[kKept];
    __shared__ float fs[4][128], ls[4][128], ms[4][128];  // per row: factors of four chunks, sums and maxima of four pairs
    // chunk n (counted over the stream) is in stage n % STG, its scores in buffer
    // n & 1; a barrier of a stage or buffer completes once per use of it, the
    // others once per chunk or pair
    __shared__ uint64_t full_k[STG], full_v[STG], empty_k[STG], empty_v[STG];
    __shared__ uint64_t s_ready[2], q_ready, p_ready[4], y_ready, l_ready[4], drained;
    __shared__ uint32_t tmem_addr;
    __shared__ int gave_up, marked;
    pdl_wait();
    pdl_launch_dependents();

    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    if (warp == kAttnWarps) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_addr)), "n"(kCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) mbar_init(&s_ready[i], 1);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&p_ready[i], 9);  // weights 4, values 1, the sums of the chunk before 4
            mbar_init(&l_ready[i], 4);
        }
        for (int i = 0; i < STG; ++i) {
            mbar_init(&full_k[i], 1);
            mbar_init(&full_v[i], 1);
            mbar_init(&empty_k[i], 1);
            mbar_init(&empty_v[i], 4);
        }
        mbar_init(&q_ready, 4);
        mbar_init(&y_ready, 1);
        mbar_init(&drained, 1);
        fence_barrier_init();
        gave_up = marked = 0;
    }
    const Cut cut = cut_sequence<CK, 1>(a, kept, sums, wsum, 0);  // (a barrier within)
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = tmem_addr;
    const uint32_t base = (smem_u32(wide_smem) + 1023u) & ~1023u;
    const uint32_t odd_p = base, in_q = odd_p + 128 * CK * 4, ring = in_q + 128 * D * 4;  // ring stage: keys, then values
    const int er = cut.er, eh = cut.eh, ec = cut.ec;
    auto is_end = [&](int r, int h, int k) { return r >= a.R || (r == er && h == eh && k >= ec); };
    const bool some = cut.any && !is_end(cut.at.r, cut.at.h, cut.c);
    auto stop_of = [&](const Pair& p) { return p.r == er && p.h == eh ? ec : p.q.c1; };  // first chunk not the stream's
    // The pair behind one whose last chunk was the stream's; false: the stream's end.
    auto follow = [&](Pair& p, int& c, int& c_stop) {
        if (c_stop != p.q.c1) return false;
        next_pair<CK>(a, kept, p);
        if (is_end(p.r, p.h, p.q.c0)) return false;
        c = p.q.c0;
        c_stop = stop_of(p);
        return true;
    };
    // A warp's wait (every lane asks: one that asks for all took 40% more time);
    // false: it ran out, in this warp or another.  The clock is looked at every
    // 64 tries, its reading takes as long as a chunk's products.
    auto wait_for = [&](uint64_t* bar, uint32_t parity) {
        bool there = false;
        unsigned long long t0 = 0;
        for (int i = 1; !there; ++i) {
            there = mbar_try_wait(bar, parity & 1u);
            if (there || (i & 63)) continue;
            const unsigned long long t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            if (*const_cast<volatile int*>(&gave_up) || t - t0 > a.wait_ns) break;
        }
        const bool done = __all_sync(0xffffffffu, there);
        if (!done && lane == 0) {
            gave_up = 1;
            atomicExch(a.fault, KQ_ERR_TIMEOUT);
        }
        return done;
    };
    // Gives a warp's part of a chunk on: what it wrote or copied to shared memory
    // to the tensor cores too, and what it read of tensor memory is read.
    auto give = [&](uint64_t* bar, uint64_t* also = nullptr) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
        if (also && lane == 0) mbar_arrive(also);
    };

    if (warp >= kAttnWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        if (warp == kAttnWarps + 3 && __any_sync(0xffffffffu, some)) {
            // ---- the products: the scores two chunks ahead of the weighted values
            auto commit = [&](uint64_t* bar) {
                asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                             : "memory");
            };
            // addresses from one lane: in uniform registers a product is issued in
            // half of the time
            const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem), ring_at = __reduce_max_sync(0xffffffffu, ring);
            auto scores = [&](uint32_t n) {
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t at = __reduce_max_sync(0xffffffffu, n);
                const uint64_t k = smem_desc(ring_at + 2 * (at % STG) * HALF, 16);
                const uint32_t to = tm + kColS + (at & 1) * kBuf;
                if (elect_one()) {
#pragma unroll
                    for (int t = TERMS - 1; t >= 0; --t)  // the small terms first
#pragma unroll
                        for (int i = 0; i < D / 16; ++i)
                            mma_tc(to, tm + kColQ + t * QT + i * 8, k + (((i / 4) * 8192 + (i % 4) * 32) >> 4), IDESC_S,
                                   t != TERMS - 1 || i != 0);
                    commit(&s_ready[at & 1]);
                    commit(&empty_k[at % STG]);
                }
                __syncwarp();
            };
            auto keys_in = [&](uint32_t n) { return wait_for(&full_k[n % STG], n / STG); };
            Pair at = cut.at;
            int c = cut.c, c_stop = stop_of(at);
            uint32_t n = 0, pair = 0;
            bool good = true;
            // (conditions by vote, so that the warp is known to stay together)
            auto all = [](bool x) { return __any_sync(0xffffffffu, x) != 0; };
            do {
                good = wait_for(&q_ready, pair++) && (!OVER || n == 0 || wait_for(&y_ready, n - 1));
                if (good && (good = keys_in(n))) scores(n);
                if (good && all(c + 1 < c_stop) && (good = keys_in(n + 1))) scores(n + 1);
                for (; good && all(c < c_stop); ++c, ++n) {
                    if (!wait_for(&p_ready[n & 3], n >> 2)) {
                        good = false;
                        break;
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t now = __reduce_max_sync(0xffffffffu, n);
                    const bool products = all(*const_cast<volatile int*>(&marked) != static_cast<int>(n) + 1);
                    const uint64_t v = smem_desc(ring_at + (2 * (now % STG) + 1) * HALF, 8192);
                    const uint32_t from = tm + kColP + (now & 1) * (TERMS * PT);
                    if (elect_one()) {
                        if (products) {
#pragma unroll
                            for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
                                for (int i = 0; i < CK / 16; ++i)
                                    mma_tc(tm, from + t * PT + i * 8, v + ((i * 2048) >> 4), IDESC_Y,
                                           t != TERMS - 1 || i != 0);
                        }
                        commit(&y_ready);
                    }
                    __syncwarp();
                    if (all(c + 2 < c_stop) && (good = keys_in(n + 2) && (!OVER || wait_for(&y_ready, n)))) scores(n + 2);
                }
            } while (good && all(follow(at, c, c_stop)));
            // nothing that was issued may run on when tensor and shared memory are
            // given back (after a wait that ran out, in any warp, nobody else has
            // waited for it)
            if (elect_one()) commit(&drained);
            __syncwarp();
            mbar_wait_drain(&drained, 0);
        } else if ((warp == kAttnWarps + 1 || warp == kAttnWarps + 2) && some) {
            // ---- copies of keys, or of values: pages in batches of 8 chunks
            // (one per lane and 16 keys), as in attn_kernel
            const bool lv = warp == kAttnWarps + 1;
            const uint16_t* const pool = static_cast<const uint16_t*>(lv ? a.v : a.k);
            uint64_t *const full = lv ? full_v : full_k, *const empty = lv ? empty_v : empty_k;
            Pair lp = cut.at, np;
            int lc = cut.c, lb = lc, le, page, nb = 0, ne = 0, npage = 0;
            auto batch_end = [&](const Pair& p, int k) { return min(stop_of(p), k + 8); };
            auto pages_of = [&](const Pair& p, int k, int e) {
                const int key = k * CK + lane * 16;
                const bool seen = key < e * CK && key < p.q.len && key + 16 > window_start(a, p.q.len - (p.q.n - 1));
                return seen ? a.table[p.r * a.table_ld + (key >> a.shift)] : 0;
            };
            auto find_next = [&] {
                np = lp;
                nb = le;
                if (le == lp.q.c1) {
                    next_pair<CK>(a, kept, np);
                    nb = np.q.c0;
                }
                ne = nb;
                if (!is_end(np.r, np.h, nb)) {
                    ne = batch_end(np, nb);
                    npage = pages_of(np, nb, ne);
                }
            };
            le = batch_end(lp, lb);
            page = pages_of(lp, lb, le);
            find_next();
            // 16-byte pieces per row, rows per instruction, instructions per 16 rows
            constexpr int XR = D / 8, RPI = 32 / XR, IPH = 16 / RPI;
            const int x = lane % XR, row0 = lane / XR;
            const int lane_src = row0 * D + x * 8;
            uint32_t n = 0;
            bool good = true;
            auto hand = [&](uint32_t m) {
                if (a.test_hold == static_cast<int>(m) + 1 && !lv && blockIdx.x == 0) return;
                give(&full[m % STG], lv ? &p_ready[m & 3] : nullptr);
            };
            for (; good && lc < le; ++n) {
                if (n >= STG && !wait_for(&empty[n % STG], n / STG - 1)) {
                    good = false;
                    break;
                }
                const int k0 = lc * CK, hi = lp.q.len, lo = window_start(a, hi - (lp.q.n - 1));
                const uint32_t to = ring + (2 * (n % STG) + (lv ? 1 : 0)) * HALF + (x >> 3) * 8192 + row0 * 128;
                const int64_t in_pool = static_cast<int64_t>(lp.h << a.shift) * D + lane_src;
                const uint16_t* src[4];
                bool ok[4];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int pg = __shfl_sync(0xffffffffu, page, 4 * (lc - lb) + h);
                    ok[h] = pg >= 0 && pg < a.n_pages;
                    src[h] = pool + (ok[h] ? pg : 0) * a.page_stride + in_pool + ((k0 + 16 * h) & ((1 << a.shift) - 1)) * D;
                }
                const bool fine = ok[0] && ok[1] && ok[2] && ok[3];
                if (!fine && a.status && lane == 0) *a.status = KQ_ERR_DEVICE_CHECK;
                if (fine && k0 >= lo && k0 + CK <= hi) {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll
                        for (int i = 0; i < IPH; ++i)
                            copy16(to + h * 2048 + i * RPI * 128 + (((x & 7) ^ ((i * RPI + row0) & 7)) << 4),
                                   src[h] + i * RPI * D, true);
                } else {
#pragma unroll
                    for (int h = 0; h < 4; ++h)
#pragma unroll 1
                        for (int i = 0; i < IPH; ++i) {
                            const int key = k0 + 16 * h + i * RPI + row0;
                            const bool in = ok[h] && key >= lo && key < hi;
                            copy16(to + h * 2048 + i * RPI * 128 + (((x & 7) ^ ((i * RPI + row0) & 7)) << 4),
                                   in ? static_cast<const void*>(src[h] + i * RPI * D) : a.k, in);
                        }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
                // three chunks on their way (handing the second last on before the wait
                // for a stage, or all three then, took 3% to 25% more time)
                if (n >= 2) {
                    asm volatile("cp.async.wait_group 2;" ::: "memory");
                    hand(n - 2);
                }
                if (++lc == le) {
                    lp = np;
                    lb = lc = nb;
                    le = ne;
                    page = npage;
                    if (lc < le) find_next();
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            if (good && n >= 2) hand(n - 2);
            if (good && n >= 1) hand(n - 1);
        }
    } else if (warp < 4) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        // ---- softmax: a thread has a row
        const int row = tid;
        const uint32_t tmem_lane = tmem + (static_cast<uint32_t>(32 * warp) << 16);
        const uint32_t my_p = odd_p + row * CK * 4;
        Pair at = cut.at;
        int c = cut.c, c_stop = some ? stop_of(at) : 0;
        bool good = some;
        uint32_t n = 0, pair = 0;
        const uint32_t my_q = in_q + warp * 128 * D, my_row = my_q + lane * 4 * D;
        // A pair's queries to shared memory, a warp its rows together; 16-byte
        // pieces at their place ^ (row & 7).  Loops are rolled: instructions that
        // run once per pair come slowly (straight through, this and the terms took
        // 20000 cycles).
        auto load_queries = [&](const Pair& p) {
            const int rows = p.q.n * a.G;
            if (32 * warp < rows) {
                const int tok = row < rows ? column_of(a, row) : 0, head = row < rows ? p.h * a.G + row - tok * a.G : 0;
                const float* const src = a.q + (p.q.first + tok) * a.ldq + static_cast<int64_t>(head) * D;
#pragma unroll 4
                for (int j = 0; j < 32; ++j) {
                    const unsigned long long row_at = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), j);
                    const float* const from = reinterpret_cast<const float*>(row_at) + 2 * lane;
                    const bool in = 32 * warp + j < rows;
#pragma unroll
                    for (int h = 0; h < D; h += 64) {
                        const uint32_t to = my_q + j * 4 * D + (((h + 2 * lane) >> 2 ^ (j & 7)) << 4) + (lane & 1) * 8;
                        if (a.vec) {
                            copy_small<8>(to, from + h, in);
                        } else {
                            copy_small<4>(to, from + h, in);
                            copy_small<4>(to + 4, from + h + 1, in);
                        }
                    }
                }
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        if (good) load_queries(at);
        while (good) {
            Pair next = at;
            int next_c = c, next_stop = c_stop;
            const bool more = follow(next, next_c, next_stop);
            const int rows = at.q.n * a.G;
            const bool live = 32 * warp < rows, mine = row < rows;
            const int tok = mine ? column_of(a, row) : at.q.n - 1;  // (a lane without a row keeps to the last one's keys)
            const int row_hi = at.q.len - (at.q.n - 1 - tok), row_lo = window_start(a, row_hi);
            float m = kNoBound, l = 0.f, dn = 1.f;
            if (live) {
                // the queries' terms
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                __syncwarp();
                auto four_at = [&](int i) {
                    const uint4 w = ld_s128(my_row + ((i ^ (lane & 7)) << 4));
                    return make_float4(__uint_as_float(w.x) * a.scale, __uint_as_float(w.y) * a.scale,
                                       __uint_as_float(w.z) * a.scale, __uint_as_float(w.w) * a.scale);
                };
                float mx = 0.f;
#pragma unroll 8
                for (int i = 0; i < D / 4; ++i) {
                    const float4 x = four_at(i);
                    mx = fmaxf(fmaxf(mx, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
                }
                int e = (__float_as_int(mx) >> 23) - 127;
                e = mx > 0.f && mx < INFINITY ? min(max(e, -100), TGT + 126) : TGT;  // (up is 2^-126 at least)
                const float up = __int_as_float((TGT - e + 127) << 23);
                dn = __int_as_float((e - TGT + 127) << 23);
#pragma unroll 1
                for (int h = 0; h < D; h += 32) {
                    uint32_t w[TERMS][16];
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        float4 x = four_at((h + 2 * j) / 4);
                        x.x *= up, x.y *= up, x.z *= up, x.w *= up;
#pragma unroll
                        for (int t = 0; t < TERMS; ++t) {
                            w[t][j] = take_term<BF16>(x.x, x.y);
                            w[t][j + 1] = take_term<BF16>(x.z, x.w);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < TERMS; ++t) tmem_store16(tmem_lane + kColQ + t * QT + h / 2, w[t]);
                }
                __syncwarp();
            }
            give(&q_ready);
            if (more) load_queries(next);

            // pages that are not in the pool, lane i & 3 for 16 keys of the next chunk
            auto page_of = [&](int k) {
                const int key = k * CK + 16 * (lane & 3);
                const bool seen = k < c_stop && key < at.q.len && key + 16 > window_start(a, at.q.len - (at.q.n - 1));
                return seen ? a.table[at.r * a.table_ld + (key >> a.shift)] : 0;
            };
            int page = page_of(c);
            for (; c < c_stop; ++c, ++n) {
                const int k0 = c * CK;
                const int bad = __ballot_sync(0xffffffffu, page < 0 || page >= a.n_pages) & 15;
                page = page_of(c + 1);
                if (!wait_for(&s_ready[n & 1], n >> 1)) {
                    good = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                float s[CK];
                uint32_t seen[2] = {0xffffffffu, 0xffffffffu};  // a bit per key
                if (k0 < row_lo || k0 + CK > row_hi || bad) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int lo = min(max(row_lo - k0 - 32 * h, 0), 32), hi = min(max(row_hi - k0 - 32 * h, 0), 32);
                        seen[h] = static_cast<uint32_t>((1ull << hi) - 1) & ~static_cast<uint32_t>((1ull << lo) - 1);
                        if (bad >> (2 * h) & 1) seen[h] &= 0xffff0000u;
                        if (bad >> (2 * h + 1) & 1) seen[h] &= 0xffffu;
                    }
                }
                if (live) {
#pragma unroll
                    for (int h = 0; h < CK; h += 32) {
                        float x[32];
                        tmem_load32(x, tmem_lane + kColS + (n & 1) * kBuf + h);
#pragma unroll
                        for (int i = 0; i < 32; ++i) s[h + i] = x[i];
                    }
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
                    if ((seen[0] & seen[1]) != 0xffffffffu) {
#pragma unroll
                        for (int i = 0; i < CK; ++i)
                            if (!(seen[i >> 5] >> (i & 31) & 1)) s[i] = -INFINITY;
                    }
                    float v0 = s[0], v1 = s[1];
#pragma unroll
                    for (int i = 2; i < CK; i += 2) v0 = fmaxf(v0, s[i]), v1 = fmaxf(v1, s[i + 1]);
                    const float mn = fmaxf(m, bound_of<BF16>(fmaxf(v0, v1) * dn));
                    const float f = ex2(m - mn);
                    m = mn;
                    fs[n & 3][row] = f;
                    float sum[2] = {0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < CK; ++i) {
                        s[i] = ex2(fmaf(s[i], dn, -mn));
                        sum[i & 1] += s[i];
                    }
                    l = fmaf(l, f, sum[0] + sum[1]);
                }
                // keys that some rows see and others do not, with values that are not
                // all finite: key by key, each row only what it sees, as in attn_kernel
                const int len = at.q.len, n1 = at.q.n - 1;
                if (min(len, k0 + CK) > len - n1 || max(window_start(a, len - n1), k0) < window_start(a, len)) {
                    const uint32_t values = ring + (2 * (n % STG) + 1) * HALF;
                    if (!wait_for(&full_v[n % STG], n / STG) ||
                        (n > 0 && !wait_for(&empty_v[(n - 1) % STG], (n - 1) / STG))) {
                        good = false;
                        break;
                    }
                    bool found = false;
                    for (uint32_t i = tid * 16; i < HALF; i += 128 * 16) {
                        const uint4 v = ld_s128(values + i);
                        found = found || not_finite<BF16>(v.x) || not_finite<BF16>(v.y) || not_finite<BF16>(v.z) ||
                                not_finite<BF16>(v.w);
                    }
                    if (found) marked = static_cast<int>(n) + 1;
                    if (live) {
#pragma unroll
                        for (int i = 0; i < CK; i += 4) {
                            const uint32_t to = my_p + ((i >> 2 ^ (row & 7)) << 4);
#pragma unroll
                            for (int k = 0; k < 4; ++k) st_s32f(to + 4 * k, seen[i >> 5] >> (i + k & 31) & 1 ? s[i + k] : -1.f);
                        }
                    }
                }
                if (live) {
#pragma unroll
                    for (int h = 0; h < CK / 2; h += 16) {
                        uint32_t w[TERMS][16];
#pragma unroll
                        for (int j = 0; j < 16; ++j)
#pragma unroll
                            for (int t = 0; t < TERMS; ++t) w[t][j] = take_term<BF16>(s[2 * (h + j)], s[2 * (h + j) + 1]);
#pragma unroll
                        for (int t = 0; t < TERMS; ++t) tmem_store16(tmem_lane + kColP + (n & 1) * (TERMS * PT) + t * PT + h, w[t]);
                    }
                }
                give(&p_ready[n & 3]);
            }
            if (!good) break;
            ls[pair & 3][row] = l;
            ms[pair & 3][row] = m;
            give(&l_ready[pair & 3]);
            ++pair;
            at = next;
            c = next_c;
            c_stop = next_stop;
            good = more;
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
        // ---- sums: a thread has a row
        const int row = tid - 128;
        const uint32_t tmem_lane = tmem + (static_cast<uint32_t>(32 * (warp - 4)) << 16);
        const uint32_t my_p = odd_p + row * CK * 4;
        float* const block_part = a.part + static_cast<int64_t>(blockIdx.x) * a.tiles * 3 * PF;
        Pair at = cut.at;
        int c = cut.c, c_stop = some ? stop_of(at) : 0;
        int64_t seg0 = cut.seg0;
        bool began = c > at.q.c0, good = some;
        uint32_t n = 0, pair = 0;
        give(&p_ready[0]);
        int4 cont = make_int4(0, 0, 0, 0);  // the pair that continues in later blocks, if it began in this one
        int cont_last = 0;
        while (good) {
            const int rows = at.q.n * a.G;
            const bool live = 32 * (warp - 4) < rows;
            float o[D];
#pragma unroll
            for (int i = 0; i < D; ++i) o[i] = 0.f;
            for (; c < c_stop; ++c, ++n) {
                if (!wait_for(&p_ready[n & 3], n >> 2) || !wait_for(&y_ready, n)) {
                    good = false;
                    break;
                }
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                if (live) {
                    const float f = *const_cast<volatile float*>(&fs[n & 3][row]);
                    if (*const_cast<volatile int*>(&marked) != static_cast<int>(n) + 1) {
#pragma unroll
                        for (int h = 0; h < D; h += 32) {
                            float y[32];
                            tmem_load32(y, tmem_lane + h);
                            asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[h + i] = fmaf(o[h + i], f, y[i]);
                        }
                    } else {
                        const uint32_t values = ring + (2 * (n % STG) + 1) * HALF;
#pragma unroll
                        for (int i = 0; i < D; ++i) o[i] *= f;
#pragma unroll 1
                        for (int k = 0; k < CK; ++k) {
                            const float p = ld_s32f(my_p + ((k >> 2 ^ (row & 7)) << 4) + (k & 3) * 4);
                            if (p < 0.f) continue;  // not the row's
#pragma unroll
                            for (int i = 0; i < D; i += 2) {
                                const float2 u = unpack<BF16>(
                                    ld_s32(values + (i >> 6) * 8192 + k * 128 + (((i >> 3 & 7) ^ (k & 7)) << 4) + (i & 6) * 2));
                                o[i] = fmaf(p, u.x, o[i]);
                                o[i + 1] = fmaf(p, u.y, o[i + 1]);
                            }
                        }
                    }
                }
                give(&empty_v[n % STG], &p_ready[(n + 1) & 3]);
            }
            if (!good || !wait_for(&l_ready[pair & 3], pair >> 2)) break;

            // ---- the pair ends here, or the stream does
            const bool ends = c_stop == at.q.c1;
            if (row < rows) {
                const float m = *const_cast<volatile float*>(&ms[pair & 3][row]);
                const float L = *const_cast<volatile float*>(&ls[pair & 3][row]);
                if (ends && !began) {
                    const int tok = column_of(a, row);
                    float* dst = a.out + (at.q.first + tok) * a.ldo + static_cast<int64_t>(at.h * a.G + row - tok * a.G) * D;
                    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
                    for (int i = 0; i < D; i += 2) store_pair(dst + i, o[i] * inv, o[i + 1] * inv, a.vec);
                } else {
                    float* dst = block_part + ((row / TR) * 3 + (began ? 0 : 1)) * PF;
                    const int r = row % TR;
#pragma unroll
                    for (int i = 0; i < D; i += 4)
                        *reinterpret_cast<float4*>(dst + r * D + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                    dst[TR * D + r] = m;
                    dst[TR * D + TR + r] = L;
                }
            }
            const int64_t units = kPairCost + (at.q.c1 - at.q.c0);
            if (!ends && !began) {
                cont = make_int4(1, at.q.first, at.q.n, at.h);
                cont_last = static_cast<int>((seg0 + units - 1) / cut.per);
            }
            seg0 += units;
            began = false;
            ++pair;
            good = follow(at, c, c_stop);
        }
        if (row == 0) {
            a.head[2 * blockIdx.x] = cont;
            a.head[2 * blockIdx.x + 1] = make_int4(cont_last, 0, 0, 0);
        }
        asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    }
    __syncthreads();
    if (warp == kAttnWarps) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kCols));
    }
}

template <int D, bool BF16>
cudaError_t launch_attn_wide(const AttnArgs& a, int blocks, cudaStream_t s) {
    constexpr size_t smem = kWideSmem<D>;
    auto kern = attn_wide_kernel<D, BF16>;
    cudaError_t err = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
    if (err != cudaSuccess) return err;
    err = launch_pdl(kern, dim3(blocks), dim3(kWideThreads), smem, 1, s, a);
    if (err != cudaSuccess) return err;
    return launch_pdl(attn_join_kernel<D, 16>, dim3(blocks, a.tiles), dim3(256), 0, 1, s, a, 1);
}

}  // namespace kq
