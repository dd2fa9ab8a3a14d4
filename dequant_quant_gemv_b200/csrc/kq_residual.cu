// kq_residual.cu — the step after a block: routed rows summed, norm, gate,
// scale, residual, and the norm in front of the next block, in one pass.
#include "kq_device.cuh"
#include "kq_layer.h"

namespace kq {

constexpr int kShortColumns = 4;  // short columns per block

struct ResidualArgs {
    int64_t T, N, slice;  // floats of a column, and of a block's part of it
    int csize;         // blocks (a cluster) per column
    kq_residual r;
};

// Sum of v over the column: over the warp (ONE), over the block, and over the cluster's blocks
// where a column has several (each warp's sum goes to every block's buffer;
// all add them in the same order).  buf: 8 * 32 floats, used once.  `started`:
// the cluster's blocks are known to run.  Another block's shared memory may
// not be touched before that, so every thread has arrived at the cluster's
// barrier when it began, and waits for the others here, behind its loads.
template <bool ONE>
__device__ __forceinline__ float column_sum(float v, float* buf, int csize, int rank, bool& started) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (ONE) return v;
    if (csize == 1) {
        if (lane == 0) buf[warp] = v;
        __syncthreads();
    } else {
        if (!started) cluster_wait();
        started = true;
        if (lane < csize) st_cluster_f32(map_rank(smem_u32(buf + rank * nw + warp), lane), v);
        cluster_sync();
    }
    float s = 0.f;
    for (int i = lane; i < csize * nw; i += 32) s += buf[i];
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// A block holds its part of one column in registers (VPT float4 per thread)
// from the first load to the last store, so every value is read and written
// once; the two norms cost one reduction each.  Few columns are split over
// the blocks of a cluster, whose sums meet in shared memory.  Bound by the
// bytes for many columns, by load latency and the two reductions for few.
// 2048 columns of eight routed rows of 2048: 34 us, 5.9 TB/s, 90% of a copy; one
// column of 4096: 2.3 us, and no more than without the wait for the cluster's
// start.  Short columns take a warp each (ONE): 60000 columns of 100 take 19 us,
// and took 62 with a block each.
template <bool VEC, int VPT, bool ONE>
__global__ void __launch_bounds__(ONE ? 32 * kShortColumns : 1024) residual_kernel(ResidualArgs a) {
    __shared__ float buf[2][8 * 32];
    bool started = ONE || a.csize == 1;
    if (!started) cluster_arrive();
    pdl_wait();
    pdl_launch_dependents();
    const kq_residual& r = a.r;
    const int rank = a.csize > 1 ? static_cast<int>(blockIdx.x % a.csize) : 0;
    const int64_t t = ONE           ? static_cast<int64_t>(blockIdx.x) * kShortColumns + (threadIdx.x >> 5)
                      : a.csize > 1 ? blockIdx.x / a.csize
                                    : blockIdx.x;
    if (ONE && t >= a.T) return;
    const int first = ONE ? threadIdx.x & 31 : threadIdx.x;
    const int base = static_cast<int>(rank * a.slice);
    const int len = static_cast<int>(min(a.slice, a.N - base));  // may be < 1 for a last block
    const int TPB = ONE ? 32 : blockDim.x;
    constexpr int W = VEC ? 4 : 1;            // floats per access
    constexpr int A = VEC ? VPT : 4 * VPT;    // accesses per thread

    auto index = [&](int i) { return W * (first + i * TPB); };
    auto load = [&](const float* p, float (&v)[A * W]) {
#pragma unroll
        for (int i = 0; i < A; ++i) {
            const int e = index(i);
            if constexpr (VEC) {
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (e < len) f = *reinterpret_cast<const float4*>(p + base + e);
                v[4 * i] = f.x, v[4 * i + 1] = f.y, v[4 * i + 2] = f.z, v[4 * i + 3] = f.w;
            } else {
                v[i] = e < len ? p[base + e] : 0.f;
            }
        }
    };
    auto store = [&](float* p, const float (&v)[A * W]) {
#pragma unroll
        for (int i = 0; i < A; ++i) {
            const int e = index(i);
            if (e >= len) continue;
            if constexpr (VEC) *reinterpret_cast<float4*>(p + base + e) = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            else p[base + e] = v[i];
        }
    };

    float o[A * W], tmp[A * W];
#pragma unroll
    for (int i = 0; i < A * W; ++i) o[i] = 0.f;
    if (r.n_terms > 0) {
        const float* y = r.y + t * r.ldy;
        float s[A * W];
        if (!r.weights && r.n_terms == 1) {
            load(y, s);
        } else {
#pragma unroll
            for (int i = 0; i < A * W; ++i) s[i] = 0.f;
#pragma unroll 8
            for (int j = 0; j < r.n_terms; ++j) {
                const float w = r.weights ? r.weights[t * r.ldw + j] : 1.f;
                load(y + j * r.ld_term, tmp);
#pragma unroll
                for (int i = 0; i < A * W; ++i) s[i] = fmaf(w, tmp[i], s[i]);
            }
        }
        if (r.res) load(r.res + t * r.ldres, o);
        float k = r.scale;
        if (r.post_gamma) {
            load(r.post_gamma, tmp);
            float sq = 0.f;
#pragma unroll
            for (int i = 0; i < A * W; ++i) sq = fmaf(s[i], s[i], sq);
            const float m = column_sum<ONE>(sq, buf[0], a.csize, rank, started) / static_cast<float>(a.N) + r.eps;
            k *= rsqrtf(m);
#pragma unroll
            for (int i = 0; i < A * W; ++i) s[i] *= tmp[i];
        }
        if (r.gate) {
            load(r.gate + t * r.ldg, tmp);
#pragma unroll
            for (int i = 0; i < A * W; ++i) s[i] *= tmp[i];
        }
#pragma unroll
        for (int i = 0; i < A * W; ++i) o[i] = fmaf(k, s[i], o[i]);
    } else if (r.res) {
        load(r.res + t * r.ldres, o);
    }
    if (r.out) store(r.out + t * r.ldout, o);
    if (r.h) {
        load(r.pre_gamma, tmp);
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < A * W; ++i) sq = fmaf(o[i], o[i], sq);  // (past the part's end: zeros)
        const float k = rsqrtf(column_sum<ONE>(sq, buf[1], a.csize, rank, started) / static_cast<float>(a.N) + r.eps);
#pragma unroll
        for (int i = 0; i < A * W; ++i) o[i] *= k * tmp[i];
        store(r.h + t * r.ldh, o);
    }
    if (!started) cluster_wait();  // (no norm)
}

template <bool VEC>
static cudaError_t launch_residual(const ResidualArgs& a, int64_t T, int vpt, int threads, cudaStream_t s) {
    if (threads == 0) {
        auto one = vpt == 1 ? residual_kernel<VEC, 1, true> : residual_kernel<VEC, 2, true>;
        return launch_pdl(one, dim3(static_cast<unsigned>((T + kShortColumns - 1) / kShortColumns)),
                          dim3(32 * kShortColumns), 0, 1, s, a);
    }
    auto kern = vpt == 1 ? residual_kernel<VEC, 1, false> : vpt == 2 ? residual_kernel<VEC, 2, false>
                                                                     : residual_kernel<VEC, 4, false>;
    return launch_pdl(kern, dim3(static_cast<unsigned>(T * a.csize)), dim3(threads), 0, a.csize, s, a);
}

}  // namespace kq

using namespace kq;

extern "C" {

int kq_residual_norm(const kq_residual* r, int64_t T, int64_t N, kq_stream_t stream) {
    set_last_error(KQ_OK, "");
    if (!r) return layer_fail(KQ_ERR_INVALID_ARG, "the step is NULL");
    if (T < 0 || N < 0) return layer_fail(KQ_ERR_INVALID_ARG, "T=%lld N=%lld", (long long)T, (long long)N);
    if (r->n_terms < 0) return layer_fail(KQ_ERR_INVALID_ARG, "n_terms=%d", r->n_terms);
    if (N > 131072 || r->n_terms > 256)
        return layer_fail(KQ_ERR_UNSUPPORTED, "N=%lld n_terms=%d", (long long)N, r->n_terms);
    if (T == 0 || N == 0) return KQ_OK;
    if (!r->out && !r->h) return layer_fail(KQ_ERR_INVALID_ARG, "neither out nor h");
    if (r->n_terms > 0 && (!good(r->y, 4) || r->ldy < 0 || r->ld_term < 0 || (r->n_terms > 1 && r->ld_term < N) ||
                           (T > 1 && r->ldy < N)))
        return layer_fail(KQ_ERR_INVALID_ARG, "y: NULL, misaligned, or strides below N");
    if (r->n_terms > 0 && (!aligned_to(r->weights, 4) || (r->weights && T > 1 && r->ldw < r->n_terms)))
        return layer_fail(KQ_ERR_INVALID_ARG, "weights: misaligned, or ldw below n_terms");
    if (!aligned_to(r->gate, 4) || (r->gate && r->ldg != 0 && r->ldg < N))
        return layer_fail(KQ_ERR_INVALID_ARG, "gate: misaligned, or ldg neither 0 nor at least N");
    if (!aligned_to(r->res, 4) || (r->res && T > 1 && r->ldres < N) || !aligned_to(r->out, 4) ||
        (r->out && T > 1 && r->ldout < N) || !aligned_to(r->h, 4) || (r->h && T > 1 && r->ldh < N))
        return layer_fail(KQ_ERR_INVALID_ARG, "res, out or h: misaligned, or a stride below N");
    if (!aligned_to(r->post_gamma, 4) || (r->h && !good(r->pre_gamma, 4)))
        return layer_fail(KQ_ERR_INVALID_ARG, "a gamma is NULL or misaligned");
    const bool post = r->post_gamma && r->n_terms > 0;
    if ((post || r->h) && !(r->eps > 0.f)) return layer_fail(KQ_ERR_INVALID_ARG, "eps must be positive");
    // What is written may overlap nothing that another column reads: out may
    // be res itself (each value is read by the thread that writes it).
    auto span = [&](const float* p, int64_t ld) { return p ? sizeof(float) * (static_cast<size_t>(T - 1) * ld + N) : 0; };
    const size_t ny = r->n_terms > 0 ? span(r->y, r->ldy) + sizeof(float) * static_cast<size_t>(r->n_terms - 1) * r->ld_term : 0;
    const size_t nw = r->n_terms > 0 && r->weights ? sizeof(float) * (static_cast<size_t>(T - 1) * r->ldw + r->n_terms) : 0;
    const struct {
        const float* p;
        size_t n;
    } in[] = {{r->y, ny}, {r->weights, nw}, {r->gate, span(r->gate, r->ldg)}, {r->res, span(r->res, r->ldres)},
              {r->post_gamma, post ? sizeof(float) * N : 0}, {r->pre_gamma, r->h ? sizeof(float) * N : 0}};
    const size_t no = span(r->out, r->ldout), nh = span(r->h, r->ldh);
    if (overlap(r->out, no, r->h, nh)) return layer_fail(KQ_ERR_INVALID_ARG, "out and h overlap");
    for (const auto& i : in) {
        const bool in_place = &i == &in[3] && r->out == r->res && r->ldout == r->ldres;
        if ((overlap(r->out, no, i.p, i.n) && !in_place) || overlap(r->h, nh, i.p, i.n))
            return layer_fail(KQ_ERR_INVALID_ARG, "an output overlaps an input");
    }
    int sms = 0;
    cudaError_t err = device_sms(&sms);
    if (err != cudaSuccess) return layer_fail(KQ_ERR_CUDA, "device query: %s", cudaGetErrorString(err));

    auto vec_ok = [&](const float* p, int64_t ld) { return !p || (aligned_to(p, 16) && ld % 4 == 0); };
    const bool vec = N % 4 == 0 && (r->n_terms == 0 || (vec_ok(r->y, r->ldy) && r->ld_term % 4 == 0)) &&
                     vec_ok(r->gate, r->ldg) && vec_ok(r->res, r->ldres) && vec_ok(r->out, r->ldout) &&
                     vec_ok(r->h, r->ldh) && vec_ok(r->post_gamma, 0) && vec_ok(r->pre_gamma, 0);
    ResidualArgs a{};
    a.T = T, a.N = N;
    a.r = *r;
    int64_t C = 1;
    while (C < 8 && (T * C * 2 <= sms || N / C > 16384) && N / C > 1024) C *= 2;
    while (C < 8 && N > 16384 * C) C *= 2;
    a.csize = static_cast<int>(C);
    a.slice = ((N + C - 1) / C + 3) / 4 * 4;
    // Many columns: 16 floats per thread keep enough loads on their way with
    // few threads to bring together (2048 columns of 8 rows of 2048: 34 us,
    // with 4 per thread 38 us).  Few columns: the fewest steps per thread (8
    // such columns: 4.2 us, with 16 per thread 4.7 us).
    int vpt = T * C > 2 * sms || a.slice > 8192 ? 4 : a.slice > 4096 ? 2 : 1;
    int threads = static_cast<int>((a.slice + 128 * vpt - 1) / (128 * vpt) * 32);
    if (N <= 256) {  // a warp per column
        vpt = N <= 128 ? 1 : 2;
        threads = 0;
    }
    if (T * C > INT32_MAX) return layer_fail(KQ_ERR_UNSUPPORTED, "T=%lld", (long long)T);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    err = vec ? launch_residual<true>(a, T, vpt, threads, s) : launch_residual<false>(a, T, vpt, threads, s);
    if (err != cudaSuccess) return layer_fail(KQ_ERR_CUDA, "residual launch: %s", cudaGetErrorString(err));
    return KQ_OK;
}

}  // extern "C"
