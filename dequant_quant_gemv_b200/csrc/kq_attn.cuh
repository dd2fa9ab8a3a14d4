// kq_attn.cuh — attention of the newest tokens over the paged cache.
//
// A request's query rows (its new columns times the query heads that share
// a key-value head) meet its keys in chunks of 32, with a running maximum and
// sum of the softmax.  Every key and value is used by a few rows only, so
// the cache's bytes bound the time, and the kernel is built to keep them
// coming:
//  - the chunks of all (request, key-value head) pairs are one sequence, cut
//    into equal contiguous parts, one per stream of the GPU, whatever the
//    requests' lengths; a pair that crosses a cut is joined from partial
//    results (first in the block, then by a second kernel, always in order);
//  - a stream is a warp (or the warps that hold the other rows of the same
//    pair) with a ring of its own in shared memory, filled by 16-byte
//    asynchronous copies, keys and values in turn, so a warp waits for no
//    other one until its part is done;
//  - both products run on the tensor cores (mma.sync m16n8k16: at 8 or 16
//    rows the bytes bind long before its rate does).  The queries and the
//    softmax's weights are fp32 and enter as sums of 16-bit terms, two of
//    fp16 (22 bits) or three of bf16 (24 bits); up to 8 rows the two halves
//    of the 16-row operand take two terms of the same 8 rows, so the second
//    term costs nothing.
// Measured (device time per call): one request of 131071 keys, 8 key-value heads
// of 128, f16: 91 us, 5.9 TB/s, 90% of a copy's rate; of these about 5 us pass
// before the first keys arrive and 8 after the last, in which the parts are
// joined.  517 keys: 12 us, all of it latency.  With more than 16 rows per pair
// the warps' instructions bind (840 per 32 keys and 16 rows, 192 of them
// products; 8 warps is what the registers allow): 61 us for 136 MB at 20 rows
// of bf16.  Tried there and not kept: a barrier per ring unit in place of the
// stream's, 12 warps of 168 registers, one warp of the stream copying for all;
// none was faster.  Long pairs of more than 32 rows go to kq_attn_wide.cuh.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kq_device.cuh"
#include "kq_attn.h"

namespace kq {

// A partial result: rows x D sums, then the rows' bounds (bound_of), then their sums of
// weights.  Slots per (block, tile): its first pair, begun in an earlier block;
// its last, continued in a later one; and one per stream for a pair that
// ends inside the stream after beginning before it.
template <int D, int TR>
constexpr int kPart = TR * (D + 2);

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}

// The bound of a row that has seen no key: the lowest finite value, so that it
// is above no score.
constexpr float kNoBound = -3.402823466e38f;

// What is taken off a row's scores (in powers of two) of which `top` is the
// largest: top rounded up to a whole number, any bound serves and this one's
// factors are exact; less 14 against an f16 cache, as weights up to 2^14 keep
// the small ones normal in fp16.  The difference is rounded up, so that no
// weight is above 2^14 where the scores are so large that it is not exact.
template <bool BF16>
__device__ __forceinline__ float bound_of(float top) {
    return BF16 ? ceilf(top) : __fsub_ru(ceilf(top), 14.f);
}

template <bool BF16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The next 16-bit term of (x, y), packed; what it leaves stays in x, y, exactly.
// f16: rounded, 22 bits in two terms.  bf16: cut, 8 bits each, so that three
// terms are all 24; without conversions calls of bf16 take 1% to 3% less time.
template <bool BF16>
__device__ __forceinline__ uint32_t take_term(float& x, float& y) {
    uint32_t w;
    if constexpr (BF16) {
        const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
        w = __byte_perm(a, b, 0x7632);
        x -= __uint_as_float(a & 0xffff0000u);
        y -= __uint_as_float(b & 0xffff0000u);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        w = *reinterpret_cast<const uint32_t*>(&h);
        x -= __low2float(h);
        y -= __high2float(h);
    }
    return w;
}

// Whether either of two packed 16-bit values is infinite or NaN.
template <bool BF16>
__device__ __forceinline__ bool not_finite(uint32_t w) {
    constexpr uint32_t E = BF16 ? 0x7f80u : 0x7c00u;
    return (w & E) == E || (w >> 16 & E) == E;
}

template <bool BF16>
__device__ __forceinline__ float2 unpack(uint32_t w) {
    if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// One request as an attention call sees it.
struct Request {
    int first, n, len;  // first column, columns, tokens (clamped to the table)
    int c0, c1;         // its chunks that some column sees; c0 == c1: no columns
};

// Column (of the request) of query row `row` of a pair: row / G, rows < 128.
__device__ __forceinline__ int column_of(const AttnArgs& a, int row) { return row * a.inv_g >> 16; }

// Keys before the result are out of a window that ends before key hi.
__device__ __forceinline__ int window_start(const AttnArgs& a, int hi) {
    return a.window && hi > a.window ? hi - a.window : 0;
}

template <int CK>
__device__ __forceinline__ void set_chunks(const AttnArgs& a, Request& q) {
    q.c0 = q.c1 = 0;
    if (q.n > 0) {
        q.c0 = window_start(a, q.len - (q.n - 1)) / CK;
        q.c1 = max(q.c0 + 1, (q.len + CK - 1) / CK);  // (no key at all: one chunk of none)
    }
}

template <int CK>
__device__ __forceinline__ Request request_of(const AttnArgs& a, int r, bool& bad) {
    Request q;
    q.first = r, q.n = 1;
    if (a.q_start) {
        q.first = a.q_start[r];
        const int64_t m = static_cast<int64_t>(a.q_start[r + 1]) - q.first;
        if (q.first < 0 || m < 0 || m > a.max_q || q.first + m > a.T) {
            bad = true;
            q.n = 0;
        } else {
            q.n = static_cast<int>(m);
        }
    }
    const int64_t rows = static_cast<int64_t>(a.max_pages) << a.shift;
    const int cap = static_cast<int>(rows < kMostKeys ? rows : kMostKeys);
    q.len = a.lens[r];
    if (q.len < 0 || q.len > cap) {
        bad = true;
        q.len = q.len < 0 ? 0 : cap;
    }
    set_chunks<CK>(a, q);
    return q;
}

// A (request, key-value head) pair of the sequence.
struct Pair {
    Request q;
    int r, h;
};

constexpr int kKept = 1024;  // requests kept in shared memory (more are read again where they are needed)

template <int CK>
__device__ __forceinline__ Request kept_request(const AttnArgs& a, const int3* kept, int r) {
    if (a.R > kKept) {
        bool bad;
        return request_of<CK>(a, r, bad);
    }
    const int3 k = kept[r];
    Request q{k.x, k.y, k.z, 0, 0};
    set_chunks<CK>(a, q);
    return q;
}

// The pair behind p (r = R: none).
template <int CK>
__device__ __forceinline__ void next_pair(const AttnArgs& a, const int3* kept, Pair& p) {
    if (++p.h < a.n_kv) return;
    p.h = 0;
    do {
        if (++p.r >= a.R) return;
        p.q = kept_request<CK>(a, kept, p.r);
    } while (p.q.c0 == p.q.c1);
}

// A stream's part of the sequence.
struct Cut {
    Pair at;            // the first chunk's pair
    int c;              // the first chunk
    int er, eh, ec;     // the first pair (er = R: none) and chunk that are not the stream's
    int64_t seg0, per;  // first unit of the first pair; units per stream
    bool any;           // (a part can still be empty)
};

// The sequence's length, and the part of stream `stream` of the block's S.
// A pair counts as its chunks of CK keys and kPairCost units more.  All
// threads of the block, of which the first kAttnWarps warps share the
// requests; kept, sums and wsum are shared memory.
template <int CK, int S>
__device__ __forceinline__ Cut cut_sequence(const AttnArgs& a, int3* kept, int* sums, int* wsum, int stream) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per_thread = (a.R + 255) >> 8;
    int mine = 0;
    bool bad = false;
    for (int r = tid * per_thread; r < min(a.R, (tid + 1) * per_thread); ++r) {
        const Request q = request_of<CK>(a, r, bad);
        if (q.c1 > q.c0) mine += q.c1 - q.c0 + kPairCost;
        if (a.R <= kKept) kept[r] = make_int3(q.first, q.n, q.len);
    }
    if (bad && a.status) *a.status = KQ_ERR_DEVICE_CHECK;
    int inc = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += u;
    }
    if (warp < kAttnWarps) {
        sums[tid] = inc - mine;
        if (lane == 31) wsum[warp] = inc;
    }
    __syncthreads();
    // units of one head before each warp's requests (lane w), and in all
    const int in_warp = lane < kAttnWarps ? wsum[lane] : 0;
    int warp_end = in_warp;
    for (int o = 1; o < kAttnWarps; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, warp_end, o);
        if (lane >= o) warp_end += u;
    }
    const int warp_start = lane < kAttnWarps ? warp_end - in_warp : INT32_MAX;
    const int64_t units = static_cast<int64_t>(__shfl_sync(0xffffffffu, warp_end, kAttnWarps - 1)) * a.n_kv;
    const int all = static_cast<int>(gridDim.x) * S;
    int64_t per = units < INT32_MAX - all ? static_cast<uint32_t>(units + all - 1) / static_cast<uint32_t>(all)
                                          : (units + all - 1) / all;
    per = max(per, int64_t(1));
    const int64_t u0 = min(units, (static_cast<int64_t>(blockIdx.x) * S + stream) * per);
    const int64_t u1 = min(units, u0 + per);


    Cut k{};
    k.er = a.R, k.per = per, k.any = u0 < u1;
    if (u0 < u1) {
#pragma unroll 1
        for (int end = 0; end < 2; ++end) {
            int64_t u = end ? u1 : u0;
            if (u == units) break;
            // the warp, then the thread whose requests hold the unit
            const int w = __popc(__ballot_sync(0xffffffffu, static_cast<int64_t>(warp_start) * a.n_kv <= u)) - 1;
            u -= static_cast<int64_t>(__shfl_sync(0xffffffffu, warp_start, w)) * a.n_kv;
            const int in_thread = sums[32 * w + lane];
            const int t = __popc(__ballot_sync(0xffffffffu, static_cast<int64_t>(in_thread) * a.n_kv <= u)) - 1;
            u -= static_cast<int64_t>(__shfl_sync(0xffffffffu, in_thread, t)) * a.n_kv;
            Pair p{};
            p.r = (32 * w + t) * per_thread;
            p.q = kept_request<CK>(a, kept, p.r);
            int len = p.q.c1 > p.q.c0 ? p.q.c1 - p.q.c0 + kPairCost : 0;
            while (u >= static_cast<int64_t>(len) * a.n_kv) {
                u -= static_cast<int64_t>(len) * a.n_kv;
                p.q = kept_request<CK>(a, kept, ++p.r);
                len = p.q.c1 > p.q.c0 ? p.q.c1 - p.q.c0 + kPairCost : 0;
            }
            p.h = u < INT32_MAX ? static_cast<int>(u) / len : static_cast<int>(u / len);
            const int in_pair = static_cast<int>(u - static_cast<int64_t>(p.h) * len);
            const int chunk = p.q.c0 + max(0, in_pair - kPairCost);
            if (end) {
                k.er = p.r, k.eh = p.h, k.ec = chunk;
            } else {
                k.at = p, k.c = chunk;
                k.seg0 = u0 - in_pair;
            }
        }
    }
    return k;
}

// The pair that a stream ends in.
struct Tail {
    int first, n, h, last;  // its columns, head, and the block that its last chunk is in
};

__device__ __forceinline__ void store_pair(float* p, float x, float y, bool vec) {
    if (vec) {
        *reinterpret_cast<float2*>(p) = make_float2(x, y);
    } else {
        p[0] = x;
        p[1] = y;
    }
}

template <int D, bool BF16, bool R16, int TILES>
__global__ void __launch_bounds__(32 * kAttnWarps, 1) attn_kernel(const __grid_constant__ AttnArgs a) {
    constexpr int TR = R16 ? 16 : 8;                      // rows per tile
    constexpr int TERMS = BF16 ? 3 : 2;
    constexpr int NP = R16 ? TERMS : (TERMS + 1) / 2;     // products per operand
    constexpr int RW = R16 ? 2 : 1;                       // rows per lane
    constexpr int STEPS = D / 16, NT = D / 8;
    constexpr int ROWB = 2 * D, UNIT = kChunk * ROWB;     // a unit of the ring: a chunk's keys, or its values
    constexpr bool QS = TILES > 1;                        // the queries' terms are in shared memory
    constexpr int S = kAttnWarps / TILES;                 // streams of the block
    constexpr int RINGW = QS ? kRingShared : kRingAlone; // the ring per warp
    constexpr int NU = RINGW * TILES / UNIT;              // units of a stream's ring
    constexpr int TGT = BF16 ? 0 : 14;                    // a query row's largest value in [2^TGT, 2^(TGT+1)), at the top of bf16 [2, 4)
    constexpr int PF = kPart<D, TR>;

    extern __shared__ __align__(1024) uint8_t ring_smem[];
    __shared__ int sums[kAttnWarps * 32], wsum[kAttnWarps];
    __shared__ int3 kept[kKept];
    __shared__ Tail tails[S];
    __shared__ float join_w[2 * S][TILES * TR], join_m[2 * S][TILES * TR], join_l[2 * S][TILES * TR];
    // what a stream leaves for the join: 1 its last pair began before it,
    // 2 its last pair continues behind it, 4 that pair's partial result is in
    // the ring, 8 its first pair's is in the stream's slot
    __shared__ int left[S];
    pdl_wait();
    pdl_launch_dependents();

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, c4 = lane & 3;
    const int tile = warp % TILES, stream = warp / TILES;

    if (tid < S) left[tid] = 0;
    const Cut cut = cut_sequence<kChunk, S>(a, kept, sums, wsum, stream);

    const uint32_t ring = smem_u32(ring_smem) + stream * TILES * RINGW;
    // partial results: slot (tile, 0) the block's first pair, 1 its last, 2 + s stream s's first
    float* const block_part = a.part + static_cast<int64_t>(blockIdx.x) * TILES * (2 + S) * PF;

    // results of the current pair
    float o[NT][4], m[RW], l[RW];
    // Where the stream begins and ends: the first chunk that is not the
    // stream's is ec of pair (er, eh).
    Pair at = cut.at;
    int c = cut.c;
    const int er = cut.er, eh = cut.eh, ec = cut.ec;
    const int64_t per = cut.per;
    int64_t seg0 = cut.seg0;  // first unit of the pair in hand
    auto is_end = [&](int r, int h, int k) { return r >= a.R || (r == er && h == eh && k >= ec); };
    bool began = c > at.q.c0;          // the pair in hand, in an earlier stream
    if (cut.any && !is_end(at.r, at.h, c)) {
        // ---- the copies run ahead, in batches of up to 16 chunks of a pair
        // whose pages the lanes hold (one per 16 keys); the next batch's are
        // on their way
        Pair lp = at, np;
        int lb = c, lc = c, le, page, nb = 0, ne = 0, npage = 0;
        bool lv = false;               // the next unit is the chunk's values
        uint32_t fill = ring;          // the unit to fill
        constexpr uint32_t RING = NU * UNIT;
        uint64_t badq = 0;             // per chunk (in turn) and 16 keys: a page that is not in the pool
        int bad_in = 0, bad_out = 0;
        auto batch_end = [&](const Pair& p, int k) {
            const int e = min(p.q.c1, k + 16);
            return p.r == er && p.h == eh ? min(e, ec) : e;
        };
        // (keys that no column sees need no page: those before a window may be
        // given back.  Pages of more than 16 tokens hold a whole chunk, both
        // halves are then copied from the first one's page)
        const int together = a.shift > 4 ? kChunk : 16;
        auto pages_of = [&](const Pair& p, int k, int e) {
            const int key = (k * kChunk + lane * 16) & -together;
            const bool seen =
                key < e * kChunk && key < p.q.len && key + together > window_start(a, p.q.len - (p.q.n - 1));
            return seen ? a.table[p.r * a.table_ld + (key >> a.shift)] : 0;
        };
        auto find_next = [&] {
            np = lp;
            nb = le;
            if (le == lp.q.c1) {
                next_pair<kChunk>(a, kept, np);
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
        constexpr int XR = ROWB / 16;                     // 16-byte pieces per row
        constexpr int RPI = 32 / XR;                      // rows per instruction
        constexpr int IPH = 16 / RPI;                     // instructions per 16 rows
        constexpr int IPW = 2 * IPH / TILES;              // instructions per warp
        constexpr int PER_HALF = IPH >= TILES ? IPH / TILES : 1;
        const int x = lane % XR, row0 = tile * RPI + lane / XR;  // this lane's piece and first row
        const int lane_src = row0 % 16 * D + x * 8;
        int64_t off0 = 0, off1 = 0;                       // of the chunk's halves in their pool
        int r0 = 0, r1 = 0;                               // its rows to copy
        // Fills the next unit of the ring: instruction j of the warp copies rows
        // row0 + j * TILES * RPI.  A row's pieces are exchanged by its place in 8
        // rows, so that eight rows' equal pieces lie in different banks.
        auto copy_unit = [&] {
            if (lc < le) {
                // (the values' unit is at the same place of the other pool; where
                // registers are short, found again)
                if (TILES > 1 || !lv) {
                    const int k0 = lc * kChunk;
                    const int hi = lp.q.len;
                    const int64_t in_page = (static_cast<int64_t>(lp.h << a.shift) + (k0 & ((1 << a.shift) - 1))) * D + lane_src;
                    const int pg0 = __shfl_sync(0xffffffffu, page, 2 * (lc - lb));
                    const int pg1 = __shfl_sync(0xffffffffu, page, 2 * (lc - lb) + 1);
                    const bool ok0 = pg0 >= 0 && pg0 < a.n_pages, ok1 = pg1 >= 0 && pg1 < a.n_pages;
                    off0 = (ok0 ? pg0 : 0) * a.page_stride + in_page;
                    // (pages of 16 tokens: the second half of the chunk is in another one)
                    off1 = a.shift > 4 ? off0 + 16 * D : (ok1 ? pg1 : 0) * a.page_stride + in_page;
                    const int lo = window_start(a, hi - (lp.q.n - 1));
                    r0 = lo - k0, r1 = hi - k0;
                    if (!ok0) r0 = max(r0, 16);
                    if (!ok1) r1 = min(r1, 16);
                    const uint64_t b = (ok0 ? 0ull : 1ull) | (ok1 ? 0ull : 2ull);
                    if (!lv) {
                        badq = (badq & ~(3ull << bad_in)) | (b << bad_in);
                        bad_in = (bad_in + 2) & 63;
                    }
                    if (b && a.status && lane == 0) *a.status = KQ_ERR_DEVICE_CHECK;
                }
                const uint16_t* const pool = static_cast<const uint16_t*>(lv ? a.v : a.k);
                const uint16_t *const src0 = pool + off0, *const src1 = pool + off1;
                const uint32_t to = fill + row0 * ROWB;
                if (r0 <= 0 && r1 >= kChunk) {
#pragma unroll
                    for (int j = 0; j < IPW; ++j) {
                        const bool second = IPH >= TILES ? j >= PER_HALF : row0 >= 16;
                        copy16(to + j * TILES * RPI * ROWB + ((x ^ ((row0 + j * TILES * RPI) & 7)) << 4),
                               (second ? src1 : src0) + j % PER_HALF * TILES * RPI * D, true);
                    }
                } else {
#pragma unroll 1
                    for (int j = 0; j < IPW; ++j) {
                        const int row = row0 + j * TILES * RPI;
                        const bool on = row >= r0 && row < r1;
                        const uint16_t* from = (row >= 16 ? src1 : src0) + j % PER_HALF * TILES * RPI * D;
                        copy16(to + j * TILES * RPI * ROWB + ((x ^ (row & 7)) << 4), on ? static_cast<const void*>(from) : a.k, on);
                    }
                }
                fill += UNIT;
                if (fill == ring + RING) fill = ring;
                if (lv && ++lc == le) {
                    lp = np;
                    lb = lc = nb;
                    le = ne;
                    page = npage;
                    if (lc < le) find_next();
                }
                lv = !lv;
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // The oldest unit has landed for every warp of the stream, and the
        // one before it has been read by all: refill that.
        auto next_unit = [&] {
            asm volatile("cp.async.wait_group %0;" ::"n"(NU - 2) : "memory");
            if constexpr (TILES == 1) __syncwarp();
            else named_bar_sync(1 + stream, 32 * TILES);
            copy_unit();
        };

        // the queries' terms as the products take them: in registers, or (QS)
        // in shared memory behind the ring
        uint32_t qf[NP][STEPS][4];
        uint4* const qs = reinterpret_cast<uint4*>(ring_smem + kAttnWarps * RINGW) + warp * (NP * STEPS * 32) + lane;
        int row_lo[RW], row_hi[RW], full_lo = 0, full_hi = 0;
        float dn[RW];
        bool live = false;             // this tile has rows of the pair
        uint32_t unit = ring;          // in hand
        int c_stop = 0;                // the stream leaves the pair before this chunk
        bool fresh = true, primed = false;
        for (bool stops = false; !stops; ++c) {
            if (fresh) {
                // ---- a new pair: its rows' queries as 16-bit terms
                fresh = false;
                c_stop = at.r == er && at.h == eh ? ec : at.q.c1;
                const int rows = at.q.n * a.G;
                live = tile * TR < rows;
                const int t0 = column_of(a, tile * TR), t1 = column_of(a, min(rows, tile * TR + TR) - 1);
                auto hi_of = [&](int tok) { return at.q.len - (at.q.n - 1 - tok); };
                full_hi = hi_of(t0);
                full_lo = window_start(a, hi_of(t1));
                float x[RW][STEPS][4];
#pragma unroll
                for (int w = 0; w < RW; ++w) {
                    const int row = tile * TR + g + 8 * w;
                    const bool on = row < rows;
                    const int tok = on ? column_of(a, row) : 0;
                    row_hi[w] = on ? hi_of(tok) : 0;
                    row_lo[w] = on ? window_start(a, row_hi[w]) : 0;
                    const float* src =
                        a.q + (at.q.first + tok) * a.ldq + static_cast<int64_t>(at.h * a.G + (on ? row - tok * a.G : 0)) * D;
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) {
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            const int d = 16 * s + 8 * b + 2 * c4;
                            float2 f = make_float2(0.f, 0.f);
                            if (on && live) {
                                if (a.vec) f = *reinterpret_cast<const float2*>(src + d);
                                else f = make_float2(src[d], src[d + 1]);
                            }
                            x[w][s][2 * b] = f.x;
                            x[w][s][2 * b + 1] = f.y;
                        }
                    }
                }
                if (!primed) {  // (the first queries ahead of the first keys)
                    primed = true;
                    #pragma unroll 1
                    for (int i = 0; i < NU - 1; ++i) copy_unit();
                }
#pragma unroll
                for (int w = 0; w < RW; ++w) {
                    float mx = 0.f;
#pragma unroll
                    for (int s = 0; s < STEPS; ++s)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            x[w][s][i] *= a.scale;
                            mx = fmaxf(mx, fabsf(x[w][s][i]));
                        }
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    // a power of two per row takes the queries' size out of the terms
                    int e = (__float_as_int(mx) >> 23) - 127;
                    e = mx > 0.f && mx < INFINITY ? min(max(e, -100), TGT + 126) : TGT;  // (up is 2^-126 at least)
                    const float up = __int_as_float((TGT - e + 127) << 23);
                    dn[w] = __int_as_float((e - TGT + 127) << 23);
#pragma unroll
                    for (int s = 0; s < STEPS; ++s) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[w][s][i] *= up;
#pragma unroll
                        for (int b = 0; b < 2; ++b) {
                            if constexpr (R16) {
#pragma unroll
                                for (int p = 0; p < NP; ++p) qf[p][s][2 * b + w] = take_term<BF16>(x[w][s][2 * b], x[w][s][2 * b + 1]);
                            } else {
                                qf[0][s][2 * b] = take_term<BF16>(x[w][s][2 * b], x[w][s][2 * b + 1]);
                                qf[0][s][2 * b + 1] = take_term<BF16>(x[w][s][2 * b], x[w][s][2 * b + 1]);
                                if constexpr (BF16) {
                                    qf[NP - 1][s][2 * b] = take_term<BF16>(x[w][s][2 * b], x[w][s][2 * b + 1]);
                                    qf[NP - 1][s][2 * b + 1] = 0u;
                                }
                            }
                        }
                    }
                    m[w] = kNoBound;
                    l[w] = 0.f;
                }
                if constexpr (QS) {
#pragma unroll
                    for (int p = 0; p < NP; ++p)
#pragma unroll
                        for (int t = 0; t < STEPS; ++t)
                            qs[(p * STEPS + t) * 32] = make_uint4(qf[p][t][0], qf[p][t][1], qf[p][t][2], qf[p][t][3]);
                }
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
            }

            next_unit();
            const int k0 = c * kChunk;
            const uint32_t keys = unit;
            unit += UNIT;
            if (unit == ring + RING) unit = ring;
            const int bad_now = static_cast<int>(badq >> bad_out) & 3;
            bad_out = (bad_out + 2) & 63;
            const int mi = lane >> 3, mr = lane & 7;
            float s[RW][8], f[RW];  // keys 8n + 2c, +1 of the lane's rows
            bool partly = false;    // the chunk has keys that some rows see and others do not
            if (live) {
                // ---- scores: 32 keys in four tiles of 8
                // (the tensor cores cut what they add to an accumulator: chains of
                // 32 dimensions, added up with rounding, hold the error at 2e-7; at
                // 16 rows, where instructions bind, chains of all dimensions, 5e-7)
                constexpr int FLUSH = R16 ? D / 32 : 1;
                float sc[4][4];
#pragma unroll
                for (int w = 0; w < RW; ++w)
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[w][i] = 0.f;
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    uint32_t b[4][4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        ldm4(b[n], keys + (8 * n + mr) * ROWB + (((4 * j + mi) ^ mr) << 4));
                        if (j % FLUSH == 0) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
                    }
                    // the small terms first
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            uint4 t;
                            if constexpr (QS) t = qs[(p * STEPS + 2 * j + half) * 32];
                            else t = make_uint4(qf[p][2 * j + half][0], qf[p][2 * j + half][1], qf[p][2 * j + half][2],
                                                qf[p][2 * j + half][3]);
#pragma unroll
                            for (int n = 0; n < 4; ++n) mma16<BF16>(sc[n], t.x, t.y, t.z, t.w, b[n][2 * half], b[n][2 * half + 1]);
                        }
                    if ((j + 1) % FLUSH) continue;
#pragma unroll
                    for (int n = 0; n < 4; ++n)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if constexpr (R16) {
                                s[0][2 * n + i] += sc[n][i];
                                s[1][2 * n + i] += sc[n][2 + i];
                            } else {
                                s[0][2 * n + i] += sc[n][i] + sc[n][2 + i];
                            }
                        }
                }
                if (k0 < full_lo || k0 + kChunk > full_hi || bad_now) {
                    partly = min(at.q.len, k0 + kChunk) > full_hi ||
                             max(window_start(a, at.q.len - (at.q.n - 1)), k0) < full_lo;
#pragma unroll
                    for (int w = 0; w < RW; ++w)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int key = k0 + 8 * (i >> 1) + 2 * c4 + (i & 1);
                            if (key < row_lo[w] || key >= row_hi[w] || (bad_now >> (i >> 2) & 1)) s[w][i] = -INFINITY;
                        }
                }
                // ---- running bound of the scores; the sums so far shrink where it
                // grows
#pragma unroll
                for (int w = 0; w < RW; ++w) {
                    float v = s[w][0];
#pragma unroll
                    for (int i = 1; i < 8; ++i) v = fmaxf(v, s[w][i]);
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
                    const float mn = fmaxf(m[w], bound_of<BF16>(v * dn[w]));
                    f[w] = ex2(m[w] - mn);
                    m[w] = mn;
                    float sum = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        s[w][i] = ex2(fmaf(s[w][i], dn[w], -mn));
                        sum += s[w][i];
                    }
                    l[w] = fmaf(l[w], f[w], sum);
                }
            }
            next_unit();
            const uint32_t values = unit;
            unit += UNIT;
            if (unit == ring + RING) unit = ring;
            bool odd = false;       // such a key's values are not all finite: 0 * NaN must stay out of the other rows
            if (partly) {
                for (int i = lane * 16; i < UNIT; i += 512) {
                    const uint4 v = ld_s128(values + i);
                    odd = odd || not_finite<BF16>(v.x) || not_finite<BF16>(v.y) || not_finite<BF16>(v.z) || not_finite<BF16>(v.w);
                }
                odd = __any_sync(0xffffffffu, odd);
            }
            if (odd) {
                // key by key, each row only what it sees
                float w8[RW][8];
#pragma unroll
                for (int w = 0; w < RW; ++w)
#pragma unroll
                    for (int i = 0; i < 8; ++i) w8[w][i] = s[w][i];
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[i][j] *= f[(j >> 1) * (RW - 1)];
#pragma unroll 1
                for (int k = 0; k < kChunk; ++k) {
                    float p[RW];
                    bool sees[RW];
#pragma unroll
                    for (int w = 0; w < RW; ++w) {
                        p[w] = __shfl_sync(0xffffffffu, w8[w][2 * (k >> 3) + (k & 1)], (lane & ~3) | (k >> 1 & 3));
                        sees[w] = k0 + k >= row_lo[w] && k0 + k < row_hi[w] && !(bad_now >> (k >> 4) & 1);
                    }
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        const float2 v = unpack<BF16>(ld_s32(values + k * ROWB + ((i ^ (k & 7)) << 4) + 4 * c4));
#pragma unroll
                        for (int w = 0; w < RW; ++w)
                            if (sees[w]) {
                                o[i][2 * w] = fmaf(p[w], v.x, o[i][2 * w]);
                                o[i][2 * w + 1] = fmaf(p[w], v.y, o[i][2 * w + 1]);
                            }
                    }
                }
            } else if (live) {
                // ---- weights, as terms (bf16 against 16 rows: 16 keys at a
                // time, which leaves registers for the queries' three terms)
                constexpr int TOGETHER = R16 && BF16 && !QS ? 1 : 2;
#pragma unroll
                for (int h0 = 0; h0 < 2; h0 += TOGETHER) {
                    uint32_t pf[TOGETHER][NP][4];
#pragma unroll
                    for (int k = 0; k < TOGETHER; ++k)
#pragma unroll
                        for (int w = 0; w < RW; ++w)
#pragma unroll
                            for (int n = 0; n < 2; ++n) {
                                float &p0 = s[w][4 * (h0 + k) + 2 * n], &p1 = s[w][4 * (h0 + k) + 2 * n + 1];
                                if constexpr (R16) {
#pragma unroll
                                    for (int t = 0; t < NP; ++t) pf[k][t][2 * n + w] = take_term<BF16>(p0, p1);
                                } else {
                                    pf[k][0][2 * n] = take_term<BF16>(p0, p1);
                                    pf[k][0][2 * n + 1] = take_term<BF16>(p0, p1);
                                    if constexpr (BF16) {
                                        pf[k][NP - 1][2 * n] = take_term<BF16>(p0, p1);
                                        pf[k][NP - 1][2 * n + 1] = 0u;
                                    }
                                }
                            }
                    // ---- weighted values
#pragma unroll
                    for (int i = 0; i < NT; i += 4) {
                        float y[4][4] = {};
#pragma unroll
                        for (int k = 0; k < TOGETHER; ++k) {
                            uint32_t b[2][4];
                            const int key = 16 * (h0 + k) + 8 * (mi & 1) + mr;
#pragma unroll
                            for (int q = 0; q < 2; ++q)
                                ldm4t(b[q], values + key * ROWB + (((i + 2 * q + (mi >> 1)) ^ mr) << 4));
#pragma unroll
                            for (int p = NP - 1; p >= 0; --p)
#pragma unroll
                                for (int n = 0; n < 4; ++n)
                                    mma16<BF16>(y[n], pf[k][p][0], pf[k][p][1], pf[k][p][2], pf[k][p][3],
                                                b[n >> 1][2 * (n & 1)], b[n >> 1][2 * (n & 1) + 1]);
                        }
#pragma unroll
                        for (int n = 0; n < 4; ++n)
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                o[i + n][j] = h0 ? o[i + n][j] + y[n][j] : fmaf(o[i + n][j], f[(j >> 1) * (RW - 1)], y[n][j]);
                    }
                }
            }

            // ---- the pair ends here, or the stream does
            if (c + 1 == c_stop) {
                const bool ends = c_stop == at.q.c1;
                Pair behind = at;
                if (ends) next_pair<kChunk>(a, kept, behind);
                stops = !ends || is_end(behind.r, behind.h, behind.q.c0);
                if (live) {
#pragma unroll
                    for (int w = 0; w < RW; ++w) {
                        l[w] += __shfl_xor_sync(0xffffffffu, l[w], 1);
                        l[w] += __shfl_xor_sync(0xffffffffu, l[w], 2);
                    }
                    if constexpr (!R16) {
#pragma unroll
                        for (int i = 0; i < NT; ++i) {
                            o[i][0] += o[i][2];
                            o[i][1] += o[i][3];
                        }
                    }
                    if (ends && !began) {
#pragma unroll
                        for (int w = 0; w < RW; ++w) {
                            const int row = tile * TR + g + 8 * w;
                            if (row >= at.q.n * a.G) continue;
                            const int tok = column_of(a, row);
                            float* dst = a.out + (at.q.first + tok) * a.ldo +
                                         static_cast<int64_t>(at.h * a.G + row - tok * a.G) * D + 2 * c4;
                            const float inv = l[w] == 0.f ? 0.f : 1.f / l[w];  // no key seen: zeros
#pragma unroll
                            for (int i = 0; i < NT; ++i)
                                store_pair(dst + 8 * i, o[i][2 * w] * inv, o[i][2 * w + 1] * inv, a.vec);
                        }
                    }
                }
                if (stops && (began || !ends)) {
                    if (lane == 0 && tile == 0) {
                        left[stream] |= (began ? 1 : 0) | (ends ? 0 : 2) | 4;
                        tails[stream] = Tail{at.q.first, at.q.n, at.h,
                                             static_cast<int>((seg0 + kPairCost + (at.q.c1 - at.q.c0) - 1) / per / S)};
                    }
                } else if (began) {
                    if (live) {
                        float* dst = block_part + (tile * (2 + S) + 2 + stream) * PF;
#pragma unroll
                        for (int w = 0; w < RW; ++w) {
                            const int row = g + 8 * w;
#pragma unroll
                            for (int i = 0; i < NT; ++i)
                                *reinterpret_cast<float2*>(dst + row * D + 8 * i + 2 * c4) =
                                    make_float2(o[i][2 * w], o[i][2 * w + 1]);
                            if (c4 == 0) {
                                dst[TR * D + row] = m[w];
                                dst[TR * D + TR + row] = l[w];
                            }
                        }
                    }
                    if (lane == 0 && tile == 0) left[stream] |= 8;
                }
                if (ends && !stops) {
                    seg0 += kPairCost + (at.q.c1 - at.q.c0);
                    at = behind;
                    c = at.q.c0 - 1;
                    began = false;
                    fresh = true;
                }
            }
        }
    }
    // ---- join the block's partial results.  The ring is free now; every
    // stream's last pair goes there if it is not whole.
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    float* const mine_part = reinterpret_cast<float*>(ring_smem) + warp * PF;
    if (left[stream] & 4) {
#pragma unroll
        for (int w = 0; w < RW; ++w) {
            const int row = g + 8 * w;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                *reinterpret_cast<float2*>(mine_part + row * D + 8 * i + 2 * c4) = make_float2(o[i][2 * w], o[i][2 * w + 1]);
            if (c4 == 0) {
                mine_part[TR * D + row] = m[w];
                mine_part[TR * D + TR + row] = l[w];
            }
        }
    }
    __syncthreads();

    // The parts in order: of each stream its first pair's (2s, in its slot),
    // then its last pair's (2s + 1, in the ring).  A run of parts is one pair; it
    // begins with a last pair that did not begin before its stream, or before the block.
    uint32_t flags = 0;
#pragma unroll
    for (int s = 0; s < S; ++s) flags |= static_cast<uint32_t>(left[s]) << (4 * s);
    auto has = [&](int q) { return (flags >> (4 * (q >> 1)) & (q & 1 ? 4 : 8)) != 0; };
    auto from_before = [&](int q) { return q == 0 || (q == 1 && (flags & 1)); };
    auto begins = [&](int q) { return from_before(q) || ((q & 1) && !(flags >> (4 * (q >> 1)) & 1)); };
    auto ends_run = [&](int q) { return !(q & 1) || !(flags >> (4 * (q >> 1)) & 2); };
    auto part_of = [&](int q, int tl) {
        return q & 1 ? reinterpret_cast<const float*>(ring_smem) + ((q >> 1) * TILES + tl) * PF
                     : block_part + (tl * (2 + S) + 2 + (q >> 1)) * PF;
    };
    // the weights of the parts: a thread per row
    if (tid < TILES * TR) {
        const int tl = tid / TR, row = tid % TR;
        float pm[2 * S], top[2 * S], pl[2 * S];
#pragma unroll
        for (int q = 0; q < 2 * S; ++q) {
            pm[q] = kNoBound, pl[q] = 0.f;
            if (has(q)) {
                pm[q] = part_of(q, tl)[TR * D + row];
                pl[q] = part_of(q, tl)[TR * D + TR + row];
            }
        }
        float M = kNoBound, L = 0.f;
#pragma unroll
        for (int q = 0; q < 2 * S; ++q)
            if (has(q)) top[q] = M = begins(q) ? pm[q] : fmaxf(M, pm[q]);
        bool last = true;  // of its run
#pragma unroll
        for (int q = 2 * S - 1; q >= 0; --q)
            if (has(q)) {
                if (last || ends_run(q)) M = top[q];
                top[q] = M;
                last = begins(q);
            }
#pragma unroll
        for (int q = 0; q < 2 * S; ++q)
            if (has(q)) {
                const float w = ex2(pm[q] - top[q]);
                L = begins(q) ? w * pl[q] : fmaf(w, pl[q], L);
                join_w[q][tid] = w;
                join_m[q][tid] = top[q];
                join_l[q][tid] = L;  // whole at the run's last part
            }
    }
    __syncthreads();
    // the rows, a warp each at a time
#pragma unroll 1
    for (int i = warp; i < TILES * TR; i += kAttnWarps) {
        const int tl = i / TR, row = i % TR;
        constexpr int E = D / 32;
        float acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
        int q0 = 0;
#pragma unroll
        for (int q = 0; q < 2 * S; ++q) {
            if (!has(q)) continue;
            const float* p = part_of(q, tl) + row * D + lane;
            const float w = join_w[q][i];
            if (begins(q)) q0 = q;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[e] = begins(q) ? w * p[32 * e] : fmaf(w, p[32 * e], acc[e]);
            const bool closed = ends_run(q);
            if (!closed && q != 2 * S - 1) continue;
            if (closed && !from_before(q0)) {
                const Tail& pair = tails[q0 >> 1];
                if (i >= pair.n * a.G) continue;
                const int tok = column_of(a, i);
                float* to = a.out + (pair.first + tok) * a.ldo + static_cast<int64_t>(pair.h * a.G + i - tok * a.G) * D + lane;
                const float L = join_l[q][i], inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
                for (int e = 0; e < E; ++e) to[32 * e] = acc[e] * inv;
            } else {
                float* dst = block_part + (tl * (2 + S) + (from_before(q0) ? 0 : 1)) * PF;
#pragma unroll
                for (int e = 0; e < E; ++e) dst[row * D + lane + 32 * e] = acc[e];
                if (lane == 0) {
                    dst[TR * D + row] = join_m[q][i];
                    dst[TR * D + TR + row] = join_l[q][i];
                }
            }
        }
    }
    if (tid == 0) {
        // the pair that continues in later blocks, if it began in this one
        int4 cont = make_int4(0, 0, 0, 0);
        int last = 0;
        if (!ends_run(2 * S - 1) && has(2 * S - 1)) {
            int q0 = 2 * S - 1;
            while (q0 > 0 && !begins(q0)) q0 -= 2;
            if (!from_before(q0)) {
                cont = make_int4(1, tails[q0 >> 1].first, tails[q0 >> 1].n, tails[q0 >> 1].h);
                last = tails[q0 >> 1].last;
            }
        }
        a.head[2 * blockIdx.x] = cont;
        a.head[2 * blockIdx.x + 1] = make_int4(last, 0, 0, 0);
    }
}

template <int E>
struct Lane {
    float x[E];
};

// E (2 or 4) consecutive floats of a partial result.
template <int E>
__device__ __forceinline__ Lane<E> load_row(const float* p) {
    Lane<E> r;
    if constexpr (E == 4) {
        const float4 f = *reinterpret_cast<const float4*>(p);
        r.x[0] = f.x, r.x[1] = f.y, r.x[2] = f.z, r.x[3] = f.w;
    } else {
        const float2 f = *reinterpret_cast<const float2*>(p);
        r.x[0] = f.x, r.x[1] = f.y;
    }
    return r;
}

// The pairs that continue over blocks: block x of this kernel joins the one
// that block x of the first kernel began, its own part and the first parts of
// the blocks behind it, in that order.
template <int D, int TR>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnArgs a, int streams) {
    constexpr int PF = kPart<D, TR>;
    __shared__ float wt[8][kMaxBlocks], wl[8][kMaxBlocks];
    pdl_wait();
    pdl_launch_dependents();
    const int4 head = a.head[2 * blockIdx.x];
    const int last = a.head[2 * blockIdx.x + 1].x;
    if (!head.x) return;
    const int tile = blockIdx.y;
    const int rows = min(TR, head.z * a.G - tile * TR);
    if (rows <= 0) return;
    const int n = last - static_cast<int>(blockIdx.x) + 1;
    const int64_t gap = static_cast<int64_t>(a.tiles) * (2 + streams) * PF;  // between blocks
    const float* const own = a.part + ((static_cast<int64_t>(blockIdx.x) * a.tiles + tile) * (2 + streams) + 1) * PF;
    const float* const others = own - PF;                                    // first slots: + i * gap for i > 0
    auto part_of = [&](int i) { return i ? others + i * gap : own; };
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    constexpr int E = D / 32, AHEAD = 8;
#pragma unroll 1
    for (int row = warp; row < rows; row += 8) {
        // the first parts' rows are on their way while the weights are made
        Lane<E> v[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            if (i < n) v[i] = load_row<E>(part_of(i) + row * D + lane * E);
        float M = kNoBound, L = 0.f;
#pragma unroll 1
        for (int i = lane; i < n; i += 32) {
            const float* p = part_of(i) + TR * D + row;
            wt[warp][i] = p[0];
            wl[warp][i] = p[TR];
            M = fmaxf(M, p[0]);
        }
        for (int s = 16; s; s >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, s));
#pragma unroll 1
        for (int i = lane; i < n; i += 32) {
            const float f = ex2(wt[warp][i] - M);
            L = fmaf(f, wl[warp][i], L);
            wt[warp][i] = f;
        }
        for (int s = 16; s; s >>= 1) L += __shfl_xor_sync(0xffffffffu, L, s);
        __syncwarp();
        float acc[E];
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += AHEAD) {
            Lane<E> u[AHEAD];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                u[j] = v[j];
                if (i0 + AHEAD + j < n) v[j] = load_row<E>(part_of(i0 + AHEAD + j) + row * D + lane * E);
            }
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (i0 + j < n) {
                    const float f = wt[warp][i0 + j];
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[e] = fmaf(f, u[j].x[e], acc[e]);
                }
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
        const int rr = tile * TR + row, tok = column_of(a, rr);
        float* to = a.out + (head.y + tok) * a.ldo + static_cast<int64_t>(head.w * a.G + rr - tok * a.G) * D + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) store_pair(to + e, acc[e] * inv, acc[e + 1] * inv, a.vec);
        __syncwarp();
    }
}

template <int D, bool BF16, bool R16, int TILES>
static cudaError_t launch_tiles(const AttnArgs& a, int sms, cudaStream_t s) {
    constexpr size_t smem =
        kAttnWarps * static_cast<size_t>(TILES > 1 ? kRingShared + 16 * D * 2 * (BF16 ? 3 : 2) : kRingAlone);
    auto kern = attn_kernel<D, BF16, R16, TILES>;
    cudaError_t err = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
    if (err != cudaSuccess) return err;
    err = launch_pdl(kern, dim3(sms), dim3(32 * kAttnWarps), smem, 1, s, a);
    if (err != cudaSuccess) return err;
    return launch_pdl(attn_join_kernel<D, R16 ? 16 : 8>, dim3(sms, TILES), dim3(256), 0, 1, s, a, kAttnWarps / TILES);
}

// Several tiles share a stream's ring, so theirs can be smaller per warp, and
// the queries' terms go to the shared memory that this leaves: in registers
// they held the products up.
template <int D, bool BF16>
cudaError_t launch_attn(const AttnArgs& a, int blocks, cudaStream_t s) {
    if (a.max_q * a.G <= 8) return launch_tiles<D, BF16, false, 1>(a, blocks, s);
    switch (a.tiles) {
        case 1: return launch_tiles<D, BF16, true, 1>(a, blocks, s);
        case 2: return launch_tiles<D, BF16, true, 2>(a, blocks, s);
        default: return launch_tiles<D, BF16, true, 4>(a, blocks, s);
    }
}

}  // namespace kq
