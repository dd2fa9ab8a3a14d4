// kq_attn.cu — the entry point of attention over the paged cache.
#include "kq_attn.h"
#include "kq_device.cuh"

namespace kq {

// The kernel of a call.  The requests' lengths are known on the device only:
// here it is what the pages and the window allow.
static bool wide(int rows, int64_t keys, int window) {
    if (window > 0 && window < keys) keys = window;
    return rows > kTileRows || (rows > kTileRows / 2 && keys >= kWideKeys);
}

// Tiles of rows (a power of two of warps share a stream's chunks) of a call;
// the kernel for many rows needs no more than as many.
static int tile_rows(int rows) { return rows <= 8 ? 8 : 16; }
static int tile_count(int rows) {
    const int n = (rows + tile_rows(rows) - 1) / tile_rows(rows);
    int p = 1;
    while (p < n) p <<= 1;
    return p;
}

// Blocks of a launch: one per SM.
static cudaError_t attn_blocks(int* out) {
    const cudaError_t err = device_sms(out);
    if (*out > kMaxBlocks) *out = kMaxBlocks;
    return err;
}

static size_t head_bytes(int sms) { return (2 * sizeof(int4) * sms + 255) / 256 * 256; }

static size_t workspace_of(int rows, int D, int sms) {
    const int tr = tile_rows(rows), tiles = tile_count(rows);
    return head_bytes(sms) + sizeof(float) * static_cast<size_t>(sms) * tiles * (2 + kAttnWarps / tiles) * tr * (D + 2);
}

}  // namespace kq

using namespace kq;

extern "C" {

size_t kq_kv_attn_workspace_bytes(int R, int max_q, int n_q, const kq_kv_cache* cache) {
    set_last_error(KQ_OK, "");
    if (check_cache(cache) != KQ_OK) return 0;
    const int64_t rows = static_cast<int64_t>(max_q) * (n_q / cache->n_kv);
    int sms = 0;
    if (R < 1 || max_q < 1 || n_q < 1 || rows < 1 || rows > 128 || attn_blocks(&sms) != cudaSuccess) return 0;
    return workspace_of(static_cast<int>(rows), cache->head_dim, sms);
}

int kq_kv_attn(int R, int64_t T, int max_q, int n_q, const float* q, int64_t ldq, const kq_kv_cache* cache,
               const int32_t* lens, const int32_t* q_start, const int32_t* table, int64_t table_ld, int max_pages,
               float scale, int window, float* out, int64_t ldo, void* workspace, size_t workspace_bytes,
               int32_t* status, kq_stream_t stream) {
    set_last_error(KQ_OK, "");
    const int st = check_cache(cache);
    if (st != KQ_OK) return st;
    const int n_kv = cache->n_kv, D = cache->head_dim;
    if (R < 0 || T < 0 || max_q < 1 || max_q > 8 || n_q < 1 || window < 0)
        return layer_fail(KQ_ERR_INVALID_ARG, "R=%d T=%lld max_q=%d n_q=%d window=%d", R, (long long)T, max_q, n_q,
                          window);
    if (n_q % n_kv != 0) return layer_fail(KQ_ERR_INVALID_ARG, "n_q=%d is not a multiple of n_kv=%d", n_q, n_kv);
    if (static_cast<int64_t>(n_q / n_kv) * max_q > 128)
        return layer_fail(KQ_ERR_UNSUPPORTED, "%d columns of %d query heads per key-value head: more than 128 rows",
                          max_q, n_q / n_kv);
    if (R > 8192 || T > INT32_MAX) return layer_fail(KQ_ERR_UNSUPPORTED, "R=%d T=%lld", R, (long long)T);
    const float scale2 = scale * 1.44269504088896340736f;  // the softmax is taken in powers of two
    if (!(scale2 - scale2 == 0.f)) return layer_fail(KQ_ERR_INVALID_ARG, "scale=%g is not finite times log2(e)", scale);
    if (!q_start && T != R) return layer_fail(KQ_ERR_INVALID_ARG, "T=%lld without q_start is not R=%d", (long long)T, R);
    if (R == 0 || T == 0) return KQ_OK;
    if (static_cast<int64_t>(R) * max_pages > (int64_t(1) << 35) / cache->page_size)
        return layer_fail(KQ_ERR_UNSUPPORTED, "R=%d requests of %d pages of %d tokens: more than 2^35 tokens", R, max_pages,
                          cache->page_size);
    if (!good(q, 4) || !good(out, 4) || !good(lens, 4) || !aligned_to(q_start, 4) || !good(table, 4) ||
        !aligned_to(status, 4))
        return layer_fail(KQ_ERR_INVALID_ARG, "q, out, lens and table must be non-NULL, all 4-byte aligned");
    if (max_pages < 1 || table_ld < max_pages)
        return layer_fail(KQ_ERR_INVALID_ARG, "max_pages=%d table_ld=%lld", max_pages, (long long)table_ld);
    const int64_t row = static_cast<int64_t>(n_q) * D;
    if (ldq < row || ldo < row)
        return layer_fail(KQ_ERR_INVALID_ARG, "ldq=%lld ldo=%lld below the columns", (long long)ldq, (long long)ldo);
    if (overlap(q, sizeof(float) * (static_cast<size_t>(T - 1) * ldq + row), out,
                sizeof(float) * (static_cast<size_t>(T - 1) * ldo + row)))
        return layer_fail(KQ_ERR_INVALID_ARG, "out overlaps q");
    int sms = 0;
    cudaError_t err = attn_blocks(&sms);
    if (err != cudaSuccess) return layer_fail(KQ_ERR_CUDA, "device query: %s", cudaGetErrorString(err));
    const int G = n_q / n_kv, rows = max_q * G;
    const size_t need = workspace_of(rows, D, sms);
    if (!good(workspace, 16) || workspace_bytes < need)
        return layer_fail(KQ_ERR_INVALID_ARG, "workspace of %zu bytes; %zu needed, 16-byte aligned", workspace_bytes, need);
    AttnArgs a{};
    err = fault_word(&a.fault);
    if (err != cudaSuccess) return layer_fail(KQ_ERR_CUDA, "fault word: %s", cudaGetErrorString(err));
    a.R = R, a.max_q = max_q, a.n_q = n_q, a.n_kv = n_kv, a.G = G;
    while ((1 << a.shift) < cache->page_size) ++a.shift;
    a.max_pages = max_pages, a.window = window, a.tiles = tile_count(rows);
    a.inv_g = (65536 + G - 1) / G;
    a.vec = aligned_to(q, 8) && aligned_to(out, 8) && ldq % 2 == 0 && ldo % 2 == 0;
    a.T = T, a.ldq = ldq, a.ldo = ldo, a.table_ld = table_ld, a.page_stride = cache->page_stride;
    a.n_pages = cache->n_pages;
    a.scale = scale2;
    a.q = q, a.k = cache->k, a.v = cache->v, a.lens = lens, a.q_start = q_start, a.table = table;
    a.out = out, a.status = status;
    a.head = static_cast<int4*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + head_bytes(sms));
    const bool many = wide(rows, static_cast<int64_t>(max_pages) * cache->page_size, window);
    a.wait_ns = kWaitNs;
    if (many) {
        a.tiles = (rows + 15) / 16;
        a.test_hold = take_attn_hold(&a.wait_ns);
    }
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    const bool b = cache->type == KQ_KV_BF16;
    if (many)
        err = D == 128 ? (b ? launch_attn_wide<128, true>(a, sms, s) : launch_attn_wide<128, false>(a, sms, s))
                       : (b ? launch_attn_wide<64, true>(a, sms, s) : launch_attn_wide<64, false>(a, sms, s));
    else
        err = D == 128 ? (b ? launch_attn<128, true>(a, sms, s) : launch_attn<128, false>(a, sms, s))
                       : (b ? launch_attn<64, true>(a, sms, s) : launch_attn<64, false>(a, sms, s));
    if (err != cudaSuccess) return layer_fail(KQ_ERR_CUDA, "attention launch: %s", cudaGetErrorString(err));
    return KQ_OK;
}

}  // extern "C"
