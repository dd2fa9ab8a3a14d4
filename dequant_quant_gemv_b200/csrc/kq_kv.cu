// kq_kv.cu — the paged key-value cache: the page plan of a step and the
// step from the qkv product's columns to rotated queries and a written cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kq_device.cuh"
#include "kq_layer.h"

namespace kq {

int check_cache(const kq_kv_cache* c) {
    if (!c) return layer_fail(KQ_ERR_INVALID_ARG, "cache is NULL");
    if (c->type != KQ_KV_F16 && c->type != KQ_KV_BF16)
        return layer_fail(KQ_ERR_INVALID_ARG, "unknown cache type %d", c->type);
    if (!good(c->k, 16) || !good(c->v, 16))
        return layer_fail(KQ_ERR_INVALID_ARG, "cache pools must be non-NULL and 16-byte aligned");
    if (c->n_kv < 1) return layer_fail(KQ_ERR_INVALID_ARG, "n_kv=%d", c->n_kv);
    if (c->n_kv > 65535) return layer_fail(KQ_ERR_UNSUPPORTED, "n_kv=%d", c->n_kv);
    if (c->head_dim != 64 && c->head_dim != 128)
        return layer_fail(KQ_ERR_UNSUPPORTED, "head_dim=%d (64 or 128)", c->head_dim);
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
        return layer_fail(KQ_ERR_INVALID_ARG, "page_size=%d is not a power of two from 16 to 1024", c->page_size);
    if (c->n_pages < 1 || c->n_pages > INT32_MAX)
        return layer_fail(KQ_ERR_INVALID_ARG, "n_pages=%lld", (long long)c->n_pages);
    if (c->page_stride < static_cast<int64_t>(c->n_kv) * c->page_size * c->head_dim || c->page_stride % 8 != 0 ||
        c->page_stride > INT64_MAX / 4 / c->n_pages)
        return layer_fail(KQ_ERR_INVALID_ARG, "page_stride=%lld", (long long)c->page_stride);
    return KQ_OK;
}

// ------------------------------------------------------------- page plan

struct PlanArgs {
    int R, shift, max_pages, free_cap;
    int64_t T, table_ld;
    const int32_t *lens, *add, *free_pages, *n_free;
    int32_t *table, *new_lens, *q_start, *pos, *n_left, *status;
    int64_t* slots;
};

// Threads of a block, the latter above kPlanMany requests.  With 256 / 1024 (us):
// 8 requests 3.2 / 5.0, 1024 5.8 / 6.8, 1500 6.8 / 7.6, 2048 8.0 / 8.1, 4096
// 14.8 / 10.2, 8192 25.8 / 14.8.
constexpr int kPlanThreads = 256, kPlanThreadsMany = 1024, kPlanMany = 2048;

// Largest i in [0, n) with v[i] <= x, for v[0] <= x and v ascending.
__device__ __forceinline__ int last_not_above(const int* v, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The plan is two running sums over the requests (tokens, new pages), cut
// at the first request whose sum passes T or the free pages; everything
// else is a lookup in them.  The sums are a few KB: every block makes them
// for itself in shared memory (no second launch, no waiting between
// blocks), then the blocks share the columns, pages and requests to write.
// A warp takes consecutive requests, 32 at a time.  Bound by latency:
// lengths, then the pages, then the stores: 3.1 us for 8 requests of one
// token, 4.5 us for 256 requests and 56000 columns.
__global__ void __launch_bounds__(kPlanThreadsMany) plan_kernel(PlanArgs a) {
    extern __shared__ int plan_smem[];
    int* q0 = plan_smem;             // R + 1: first column of each request
    int* p0 = plan_smem + a.R + 1;   // R + 1: first new page of each request
    __shared__ long long wt[32], wp[32];
    __shared__ int cut_t[32], cut_p[32];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
    const int ps1 = (1 << a.shift) - 1;
    int nf = *a.n_free;
    nf = nf < 0 ? 0 : nf > a.free_cap ? a.free_cap : nf;

    // tokens and pages of request r (0, 0: left out)
    auto demand = [&](int r, int& tok, int& pages) {
        const int n = a.lens[r], d = a.add[r];
        const int64_t e = static_cast<int64_t>(n) + d;
        tok = pages = 0;
        if (n < 0 || d < 0 || e > (static_cast<int64_t>(a.max_pages) << a.shift) || e > INT32_MAX) return false;
        tok = d;
        pages = static_cast<int>((e + ps1) >> a.shift) - static_cast<int>((static_cast<int64_t>(n) + ps1) >> a.shift);
        return true;
    };
    auto sum_to_here = [&](long long v) {
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        return v;
    };

    const int sets = ((a.R + 31) / 32 + nw - 1) / nw;  // of 32 requests per warp
    const int r0 = warp * sets * 32;
    long long t = 0, p = 0;
    for (int i = 0; i < sets; ++i) {
        const int r = r0 + 32 * i + lane;
        int tok = 0, pages = 0;
        if (r < a.R) demand(r, tok, pages);
        t += tok;
        p += pages;
    }
    t = sum_to_here(t);
    p = sum_to_here(p);
    if (lane == 31) {
        wt[warp] = t;
        wp[warp] = p;
    }
    __syncthreads();
    long long et = 0, ep = 0;  // before the set in hand
    for (int w = 0; w < warp; ++w) {
        et += wt[w];
        ep += wp[w];
    }
    int top_t = 0, top_p = 0;  // the served requests' sums: the largest that fit
    for (int i = 0; i < sets; ++i) {
        const int r = r0 + 32 * i + lane;
        int tok = 0, pages = 0;
        if (r < a.R) demand(r, tok, pages);
        const long long it = et + sum_to_here(tok), ip = ep + sum_to_here(pages);
        if (r < a.R) {
            q0[r] = static_cast<int>(min(it - tok, static_cast<long long>(INT32_MAX)));
            p0[r] = static_cast<int>(min(ip - pages, static_cast<long long>(INT32_MAX)));
        }
        if (tok > 0 && it <= a.T && ip <= nf) {
            top_t = static_cast<int>(it);
            top_p = static_cast<int>(ip);
        }
        et = __shfl_sync(0xffffffffu, it, 31);
        ep = __shfl_sync(0xffffffffu, ip, 31);
    }
    for (int o = 16; o; o >>= 1) {
        top_t = max(top_t, __shfl_xor_sync(0xffffffffu, top_t, o));
        top_p = max(top_p, __shfl_xor_sync(0xffffffffu, top_p, o));
    }
    if (lane == 0) {
        cut_t[warp] = top_t;
        cut_p[warp] = top_p;
    }
    __syncthreads();
    for (int w = 0; w < nw; ++w) {
        top_t = max(top_t, cut_t[w]);
        top_p = max(top_p, cut_p[w]);
    }
    for (int r = tid; r <= a.R; r += blockDim.x) {  // requests behind the cut add none
        q0[r] = r < a.R ? min(q0[r], top_t) : top_t;
        p0[r] = r < a.R ? min(p0[r], top_p) : top_p;
    }
    __syncthreads();

    const int64_t first = static_cast<int64_t>(blockIdx.x) * blockDim.x + tid;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.x;
    bool bad = false;
    for (int64_t r = first; r <= a.R; r += step) {
        a.q_start[r] = q0[r];
        if (r == a.R) {
            *a.n_left = nf - top_p;
            break;
        }
        int tok, pages;
        const bool ok = demand(static_cast<int>(r), tok, pages);
        const int got = q0[r + 1] - q0[r];
        a.new_lens[r] = a.lens[r] + got;
        if (!ok || got != tok) bad = true;
    }
    for (int64_t i = first; i < top_p; i += step) {  // new page i of the step
        const int r = last_not_above(p0, a.R, static_cast<int>(i));
        const int old = static_cast<int>((static_cast<int64_t>(a.lens[r]) + ps1) >> a.shift);
        a.table[r * a.table_ld + old + (static_cast<int>(i) - p0[r])] = a.free_pages[nf - 1 - i];
    }
    for (int64_t c = first; c < a.T; c += step) {
        int64_t slot = -1;
        int at = -1;
        if (c < top_t) {
            const int r = last_not_above(q0, a.R, static_cast<int>(c));
            const int n = a.lens[r];
            at = n + (static_cast<int>(c) - q0[r]);
            const int i = at >> a.shift;
            const int old = static_cast<int>((static_cast<int64_t>(n) + ps1) >> a.shift);
            // (another block may be entering the new pages: they come from the stack)
            const int page = i < old ? a.table[r * a.table_ld + i] : a.free_pages[nf - 1 - (p0[r] + i - old)];
            if (page >= 0) slot = (static_cast<int64_t>(page) << a.shift) + (at & ps1);
            else bad = true;
        }
        a.slots[c] = slot;
        a.pos[c] = at;
    }
    if (bad && a.status) *a.status = KQ_ERR_DEVICE_CHECK;
}

// ---------------------------------------------------------------- append

struct AppendArgs {
    int64_t T, ld, ldq, page_stride, n_slots;
    int n_q, n_kv, shift, per_warp, groups;
    int rot_dim, adjacent, vec;
    float eps;
    const float *qkv, *inv_freq, *q_gamma, *k_gamma;
    const int64_t* slots;
    const int32_t* pos;
    float* q_out;
    void *k, *v;
    int32_t* status;
};

template <int E>
struct Lane {
    float x[E];
};

template <int E>
__device__ __forceinline__ Lane<E> load_lane(const float* p, bool vec) {
    Lane<E> r;
    if constexpr (E == 4) {
        if (vec) {
            const float4 f = *reinterpret_cast<const float4*>(p);
            r.x[0] = f.x, r.x[1] = f.y, r.x[2] = f.z, r.x[3] = f.w;
            return r;
        }
    } else {
        if (vec) {
            const float2 f = *reinterpret_cast<const float2*>(p);
            r.x[0] = f.x, r.x[1] = f.y;
            return r;
        }
    }
#pragma unroll
    for (int e = 0; e < E; ++e) r.x[e] = p[e];
    return r;
}

template <int E>
__device__ __forceinline__ void store_lane(float* p, const Lane<E>& r, bool vec) {
    if (vec) {
        if constexpr (E == 4) *reinterpret_cast<float4*>(p) = make_float4(r.x[0], r.x[1], r.x[2], r.x[3]);
        else *reinterpret_cast<float2*>(p) = make_float2(r.x[0], r.x[1]);
        return;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) p[e] = r.x[e];
}

template <int E, bool BF16>
__device__ __forceinline__ void store_cache(void* pool, int64_t at, const Lane<E>& r) {
    uint32_t w[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        if constexpr (BF16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(r.x[e], r.x[e + 1]);
            w[e / 2] = *reinterpret_cast<const uint32_t*>(&b);
        } else {
            const __half2 h = __floats2half2_rn(r.x[e], r.x[e + 1]);
            w[e / 2] = *reinterpret_cast<const uint32_t*>(&h);
        }
    }
    uint16_t* p = static_cast<uint16_t*>(pool) + at;
    if constexpr (E == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
}

// 4096 columns of 64 + 2*8 heads of 128: 54.8 us with 4 warps per block and 4
// heads at a time (5.8 TB/s, 89% of a copy); 8 warps 59, 2 heads 59, 8 heads 61.
constexpr int kAppendWarps = 4;
constexpr int kHeadsTogether = 4, kHeadsPerWarp = 16;

// A warp takes per_warp consecutive heads of one column, a lane E = D/32
// consecutive dimensions: a pair's partner is in the lane itself (adjacent)
// or one shuffle away (half).  The angles' sines and cosines, most of the
// arithmetic, are made once for the warp's heads.  Bound by the bytes of
// qkv, q_out and the cache for many columns, by latency for few (one column
// of 32 + 2*8 heads: 2.0 us).
template <int E, bool BF16, int HEADS>
__global__ void __launch_bounds__(32 * kAppendWarps) append_kernel(AppendArgs a) {
    constexpr int D = 32 * E;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t w = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
    const int64_t t = w / a.groups;
    if (t >= a.T) return;
    const int64_t slot = a.slots[t];
    if (slot < 0) return;
    const int heads = a.n_q + 2 * a.n_kv;
    const int h0 = static_cast<int>(w - t * a.groups) * a.per_warp;
    const int h1 = min(heads, h0 + a.per_warp);
    const bool fits = slot < a.n_slots;
    if (!fits && a.status && lane == 0) *a.status = KQ_ERR_DEVICE_CHECK;
    const int64_t page = slot >> a.shift;
    const int at = static_cast<int>(slot & ((1 << a.shift) - 1));
    const int d0 = lane * E;                    // this lane's first dimension
    const bool vec = a.vec != 0;

    float c[E], s[E];
    int partner = lane;                         // half pairing: the lane with the pair's other half
    bool turns = false, second = false;
    const bool adj = a.adjacent != 0;
    const int rot = a.rot_dim;
    if (d0 < rot && h0 < a.n_q + a.n_kv) {
        turns = true;
        const int half = rot / 2;
        second = !adj && d0 >= half;
        const double p = static_cast<double>(a.pos[t]);
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int f = adj ? (d0 + e) >> 1 : (d0 + e) - (second ? half : 0);
            // the angle in turns: the product has at most 55 bits and is
            // reduced to one turn before it is rounded to fp32
            const double turn = p * static_cast<double>(a.inv_freq[f]) * 0.15915494309189533577;
            sincospif(static_cast<float>(2.0 * (turn - rint(turn))), &s[e], &c[e]);
        }
        if (!adj) partner = second ? lane - half / E : lane + half / E;
    }
    const float* col = a.qkv + t * a.ld + d0;
    // HEADS at a time: their loads are on their way together
    for (int hb = h0; hb < h1; hb += HEADS) {
        Lane<E> xs[HEADS];
#pragma unroll
        for (int i = 0; i < HEADS; ++i)
            if (hb + i < h1) xs[i] = load_lane<E>(col + static_cast<int64_t>(hb + i) * D, vec);
#pragma unroll
        for (int i = 0; i < HEADS; ++i) {
            const int h = hb + i;
            if (h >= h1) break;
            Lane<E> x = xs[i];
            if (h >= a.n_q + a.n_kv) {
                if (fits)
                    store_cache<E, BF16>(a.v, page * a.page_stride +
                                                  (static_cast<int64_t>(h - a.n_q - a.n_kv) << a.shift) * D + at * D + d0, x);
                continue;
            }
            const float* gamma = h < a.n_q ? a.q_gamma : a.k_gamma;
            if (gamma) {
                float sq = 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) sq += x.x[e] * x.x[e];
                for (int o = 16; o; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
                const float r = rsqrtf(sq * (1.0f / D) + a.eps);
                const Lane<E> g = load_lane<E>(gamma + d0, false);
#pragma unroll
                for (int e = 0; e < E; ++e) x.x[e] *= r * g.x[e];
            }
            Lane<E> y = x;
            if (rot) {
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    const float o = adj ? x.x[e ^ 1] : __shfl_sync(0xffffffffu, x.x[e], partner);
                    const bool b = adj ? (e & 1) : second;
                    if (turns) y.x[e] = b ? o * s[e] + x.x[e] * c[e] : x.x[e] * c[e] - o * s[e];
                }
            }
            if (h < a.n_q) store_lane<E>(a.q_out + t * a.ldq + static_cast<int64_t>(h) * D + d0, y, vec);
            else if (fits)
                store_cache<E, BF16>(a.k, page * a.page_stride + (static_cast<int64_t>(h - a.n_q) << a.shift) * D + at * D + d0,
                                     y);
        }
    }
}

template <int E, bool BF16>
static auto append_of(int per_warp) {
    return per_warp == 1 ? append_kernel<E, BF16, 1> : append_kernel<E, BF16, kHeadsTogether>;
}

static int log2_of(int v) {
    int s = 0;
    while ((1 << s) < v) ++s;
    return s;
}

}  // namespace kq

using namespace kq;

extern "C" {

int kq_kv_plan(int R, const int32_t* lens, const int32_t* add, int page_size, int32_t* table, int64_t table_ld,
               int max_pages, const int32_t* free_pages, int free_cap, const int32_t* n_free, int64_t T,
               int32_t* new_lens, int32_t* q_start, int64_t* slots, int32_t* pos, int32_t* n_left, int32_t* status,
               kq_stream_t stream) {
    set_last_error(KQ_OK, "");
    if (R < 0 || T < 0 || free_cap < 0)
        return layer_fail(KQ_ERR_INVALID_ARG, "R=%d T=%lld free_cap=%d", R, (long long)T, free_cap);
    if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)))
        return layer_fail(KQ_ERR_INVALID_ARG, "page_size=%d is not a power of two from 16 to 1024", page_size);
    if (R > 8192 || T > INT32_MAX) return layer_fail(KQ_ERR_UNSUPPORTED, "R=%d T=%lld", R, (long long)T);
    if (R > 0) {
        if (!good(lens, 4) || !good(add, 4) || !good(table, 4) || !good(new_lens, 4))
            return layer_fail(KQ_ERR_INVALID_ARG, "lens, add, table and new_lens must be non-NULL and 4-byte aligned");
        if (max_pages < 1 || table_ld < max_pages)
            return layer_fail(KQ_ERR_INVALID_ARG, "max_pages=%d table_ld=%lld", max_pages, (long long)table_ld);
        const size_t n = sizeof(int32_t) * static_cast<size_t>(R);
        if (overlap(new_lens, n, lens, n) || overlap(new_lens, n, add, n))
            return layer_fail(KQ_ERR_INVALID_ARG, "new_lens overlaps lens or add");
    }
    if (free_cap > 0 && !good(free_pages, 4))
        return layer_fail(KQ_ERR_INVALID_ARG, "free_pages must be non-NULL and 4-byte aligned");
    if (!good(n_free, 4) || !good(n_left, 4) || !good(q_start, 4) || n_free == n_left)
        return layer_fail(KQ_ERR_INVALID_ARG,
                          "n_free, n_left and q_start must be non-NULL, 4-byte aligned and distinct");
    if (T > 0 && (!good(slots, 8) || !good(pos, 4)))
        return layer_fail(KQ_ERR_INVALID_ARG, "slots and pos must be non-NULL and aligned");
    if (!aligned_to(status, 4)) return layer_fail(KQ_ERR_INVALID_ARG, "status is not 4-byte aligned");
    int sms = 0;
    cudaError_t err = device_sms(&sms);
    if (err != cudaSuccess) return layer_fail(KQ_ERR_CUDA, "device query: %s", cudaGetErrorString(err));
    PlanArgs a{R, log2_of(page_size), max_pages, free_cap, T, table_ld, lens, add, free_pages, n_free,
               table, new_lens, q_start, pos, n_left, status, slots};
    const int threads = R > kPlanMany ? kPlanThreadsMany : kPlanThreads;
    const int64_t want = (T + threads - 1) / threads;
    const int grid = static_cast<int>(want < 1 ? 1 : want > sms ? sms : want);
    const size_t smem = sizeof(int) * 2 * (static_cast<size_t>(R) + 1);
    if (smem > 48 * 1024) {
        err = ensure_smem_attr(reinterpret_cast<const void*>(plan_kernel), smem);
        if (err != cudaSuccess) return layer_fail(KQ_ERR_CUDA, "shared memory: %s", cudaGetErrorString(err));
    }
    err = launch_pdl(plan_kernel, dim3(grid), dim3(threads), smem, 1, reinterpret_cast<cudaStream_t>(stream), a);
    if (err != cudaSuccess) return layer_fail(KQ_ERR_CUDA, "plan launch: %s", cudaGetErrorString(err));
    return KQ_OK;
}

int kq_kv_append(int64_t T, const float* qkv, int64_t ld, int n_q, const kq_kv_cache* cache, const int64_t* slots,
                 const int32_t* pos, const kq_rotary* rot, float* q_out, int64_t ldq, int32_t* status,
                 kq_stream_t stream) {
    set_last_error(KQ_OK, "");
    const int st = check_cache(cache);
    if (st != KQ_OK) return st;
    if (T < 0 || n_q < 1 || n_q > 65535) return layer_fail(KQ_ERR_INVALID_ARG, "T=%lld n_q=%d", (long long)T, n_q);
    const int D = cache->head_dim, n_kv = cache->n_kv, heads = n_q + 2 * n_kv;
    if (!rot) return layer_fail(KQ_ERR_INVALID_ARG, "rot is NULL");
    if (rot->rot_dim < 0 || rot->rot_dim > D || rot->rot_dim % 8 != 0)
        return layer_fail(KQ_ERR_INVALID_ARG, "rot_dim=%d is not a multiple of 8 from 0 to head_dim", rot->rot_dim);
    if (rot->rot_dim && !good(rot->inv_freq, 4))
        return layer_fail(KQ_ERR_INVALID_ARG, "inv_freq must be non-NULL and 4-byte aligned");
    if (!aligned_to(rot->q_gamma, 4) || !aligned_to(rot->k_gamma, 4))
        return layer_fail(KQ_ERR_INVALID_ARG, "gammas must be 4-byte aligned");
    if ((rot->q_gamma || rot->k_gamma) && !(rot->eps > 0.f))
        return layer_fail(KQ_ERR_INVALID_ARG, "eps must be positive");
    if (T == 0) return KQ_OK;
    if (!good(qkv, 4) || !good(q_out, 4) || !good(slots, 8) || !good(pos, 4) || !aligned_to(status, 4))
        return layer_fail(KQ_ERR_INVALID_ARG, "qkv, q_out, slots and pos must be non-NULL and aligned");
    if (ld < static_cast<int64_t>(heads) * D || ldq < static_cast<int64_t>(n_q) * D)
        return layer_fail(KQ_ERR_INVALID_ARG, "ld=%lld ldq=%lld below the columns", (long long)ld, (long long)ldq);
    const size_t nx = sizeof(float) * (static_cast<size_t>(T - 1) * ld + static_cast<size_t>(heads) * D);
    const size_t nq = sizeof(float) * (static_cast<size_t>(T - 1) * ldq + static_cast<size_t>(n_q) * D);
    if (overlap(qkv, nx, q_out, nq) && !(qkv == q_out && ld == ldq))
        return layer_fail(KQ_ERR_INVALID_ARG, "q_out overlaps qkv and is not in place");
    int sms = 0;
    cudaError_t err = device_sms(&sms);
    if (err != cudaSuccess) return layer_fail(KQ_ERR_CUDA, "device query: %s", cudaGetErrorString(err));
    AppendArgs a{};
    a.T = T, a.ld = ld, a.ldq = ldq, a.page_stride = cache->page_stride;
    a.n_slots = cache->n_pages * cache->page_size;
    a.n_q = n_q, a.n_kv = n_kv, a.shift = log2_of(cache->page_size);
    // one head per warp while that does not fill the GPU
    int64_t per = T * heads / (static_cast<int64_t>(sms) * 32);
    a.per_warp = static_cast<int>(per < 2 ? 1 : per > kHeadsPerWarp ? kHeadsPerWarp : per);
    a.groups = (heads + a.per_warp - 1) / a.per_warp;
    a.rot_dim = rot->rot_dim, a.adjacent = rot->adjacent != 0;
    a.vec = aligned_to(qkv, 16) && aligned_to(q_out, 16) && ld % 4 == 0 && ldq % 4 == 0;
    a.eps = rot->eps;
    a.qkv = qkv, a.inv_freq = rot->inv_freq, a.q_gamma = rot->q_gamma, a.k_gamma = rot->k_gamma;
    a.slots = slots, a.pos = pos, a.q_out = q_out, a.k = cache->k, a.v = cache->v, a.status = status;
    const int64_t blocks = (T * a.groups + kAppendWarps - 1) / kAppendWarps;
    if (blocks > INT32_MAX) return layer_fail(KQ_ERR_UNSUPPORTED, "T=%lld", (long long)T);
    const bool bf = cache->type == KQ_KV_BF16;
    auto kern = D == 128 ? (bf ? append_of<4, true>(a.per_warp) : append_of<4, false>(a.per_warp))
                         : (bf ? append_of<2, true>(a.per_warp) : append_of<2, false>(a.per_warp));
    err = launch_pdl(kern, dim3(static_cast<unsigned>(blocks)), dim3(32 * kAppendWarps), 0, 1,
                     reinterpret_cast<cudaStream_t>(stream), a);
    if (err != cudaSuccess) return layer_fail(KQ_ERR_CUDA, "append launch: %s", cudaGetErrorString(err));
    return KQ_OK;
}

}  // extern "C"
