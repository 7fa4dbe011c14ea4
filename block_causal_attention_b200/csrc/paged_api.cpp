// C ABI of the paged KV cache: argument checks and handle lifetime.  See include/bca.h.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "paged.hpp"

namespace {

using bca::PagedCache;

inline bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

int on_its_device(const PagedCache &c) {
    if (c.flags & BCA_PLAN_HOST_ONLY) return BCA_ERR_HOST_ONLY_PLAN;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return BCA_ERR_CUDA;
    return dev == c.device ? BCA_OK : BCA_ERR_INVALID_ARGUMENT;
}

int fill(const bca_paged_desc *d, PagedCache &c) {
    if (!d) return BCA_ERR_INVALID_ARGUMENT;
    const uint32_t known = BCA_PAGED_FP16 | BCA_O_FP32 | BCA_PLAN_HOST_ONLY | BCA_TEST_FORCE_TIMEOUT;
    if (d->flags & ~known) return BCA_ERR_INVALID_ARGUMENT;
    if (d->num_q_heads <= 0 || d->num_kv_heads <= 0 || d->num_layers <= 0 || d->num_pages <= 0)
        return BCA_ERR_INVALID_ARGUMENT;
    if (d->num_pages > INT32_MAX) return BCA_ERR_INVALID_ARGUMENT;  // tables hold int32 page numbers
    if (d->num_q_heads % d->num_kv_heads != 0) return BCA_ERR_UNSUPPORTED;
    // a KV head is a grid row of the launches
    if (d->num_kv_heads > 65535 || d->num_layers > 65535) return BCA_ERR_UNSUPPORTED;
    if (d->head_dim != 24 && d->head_dim != 32 && d->head_dim != 48) return BCA_ERR_UNSUPPORTED;
    if (!(d->norm_eps >= 0.f) || !std::isfinite(d->norm_eps)) return BCA_ERR_INVALID_ARGUMENT;
    for (float b : d->rope_base)
        if (!(b > 0.f) || !std::isfinite(b)) return BCA_ERR_INVALID_ARGUMENT;
    c.hq = d->num_q_heads;
    c.hkv = d->num_kv_heads;
    c.d = d->head_dim;
    c.layers = d->num_layers;
    c.pages = d->num_pages;
    c.eps = d->norm_eps;
    c.flags = d->flags;
    const int pairs = c.d / 2 / 3;
    for (int a = 0; a < 3; ++a)
        for (int i = 0; i < pairs; ++i) {
            const long double x = std::pow((long double)d->rope_base[a], -(long double)i / pairs) /
                                  6.283185307179586476925286766559L;
            c.turns[8 * a + i] = (uint64_t)std::ldexp(x - std::floor(x), 64);  // below 2^64
        }
    return BCA_OK;
}

}  // namespace

extern "C" {

int bca_paged_create(const bca_paged_desc *desc, bca_paged_t *out) {
    if (!out) return BCA_ERR_INVALID_ARGUMENT;
    *out = nullptr;
    bca_paged_s *h = new (std::nothrow) bca_paged_s();
    if (!h) return BCA_ERR_NO_MEMORY;
    PagedCache &c = h->cache;
    int rc = fill(desc, c);
    if (rc == BCA_OK && !(c.flags & BCA_PLAN_HOST_ONLY)) {
        if (cudaGetDevice(&c.device) != cudaSuccess) rc = BCA_ERR_CUDA;
        else if (cudaMalloc(reinterpret_cast<void **>(&c.d_status), 256) != cudaSuccess) rc = BCA_ERR_NO_MEMORY;
        else if (cudaMemset(c.d_status, 0, 256) != cudaSuccess) rc = BCA_ERR_CUDA;
        // (asynchronous, on a stream that streams made non-blocking do not wait for)
        else if (cudaStreamSynchronize(cudaStreamLegacy) != cudaSuccess) rc = BCA_ERR_CUDA;
        else rc = bca::prepare_paged(c);
    }
    if (rc != BCA_OK) {
        bca_paged_destroy(h);
        return rc;
    }
    *out = h;
    return BCA_OK;
}

void bca_paged_destroy(bca_paged_t cache) {
    if (!cache) return;
    PagedCache &c = cache->cache;
    if (c.d_status) {
        int cur = -1;
        cudaGetDevice(&cur);
        if (cur != c.device) cudaSetDevice(c.device);
        cudaFree(c.d_status);
        if (cur >= 0 && cur != c.device) cudaSetDevice(cur);
    }
    delete cache;
}

size_t bca_paged_pool_bytes(bca_paged_t cache) {
    if (!cache) return 0;
    const PagedCache &c = cache->cache;
    return (size_t)c.pages * c.hkv * bca::kPage * c.d * 2;
}

int bca_paged_write(bca_paged_t cache, const void *k, const void *v, int64_t n, const int32_t *pos,
                    const float *k_gain, const int32_t *table, int32_t seqs, int32_t width, const int32_t *off,
                    const int32_t *start, void *k_pages, void *v_pages, void *stream) {
    if (!cache || n < 0 || seqs < 0 || width < 0 || n > INT32_MAX) return BCA_ERR_INVALID_ARGUMENT;
    const PagedCache &c = cache->cache;
    int rc = on_its_device(c);
    if (rc != BCA_OK) return rc;
    if (n == 0 || seqs == 0) return BCA_OK;  // (arrays of no rows may be null)
    if (k_gain && !pos) return BCA_ERR_INVALID_ARGUMENT;
    if (!k || !v || !off || !start || !k_pages || !v_pages || (width > 0 && !table)) return BCA_ERR_INVALID_ARGUMENT;
    for (const void *p : {k, v, (const void *)k_pages, (const void *)v_pages})
        if (!aligned(p, 16)) return BCA_ERR_MISALIGNED;
    for (const void *p : {(const void *)pos, (const void *)k_gain, (const void *)table, (const void *)off,
                          (const void *)start})
        if (!aligned(p, 4)) return BCA_ERR_MISALIGNED;
    return bca::launch_paged_write(c, {k, v, n, pos, k_gain, table, seqs, width, off, start, k_pages, v_pages},
                                   static_cast<cudaStream_t>(stream));
}

int bca_paged_copy(bca_paged_t cache, const int32_t *pairs, int64_t n, void *k_pages, void *v_pages, void *stream) {
    if (!cache || n < 0) return BCA_ERR_INVALID_ARGUMENT;
    const PagedCache &c = cache->cache;
    if (n > 0 && !pairs) return BCA_ERR_INVALID_ARGUMENT;
    if (n > c.pages) return BCA_ERR_BAD_PAGE;  // some page would be written twice
    for (int64_t i = 0; i < 2 * n; ++i)
        if (pairs[i] < 0 || pairs[i] >= c.pages) return BCA_ERR_BAD_PAGE;
    try {
        // Which pages are written: a bit each (1,000 moves in a pool of 2,000 pages: 2 us), or, where
        // the pool is far larger than the call, a sorted list (the same moves: 40 us).
        if (c.pages / 64 <= 4096 + 64 * n) {
            std::vector<uint64_t> written((size_t)(c.pages / 64 + 1), 0);
            for (int64_t i = 0; i < n; ++i) {
                const uint32_t to = (uint32_t)pairs[2 * i + 1];
                const uint64_t bit = 1ull << (to % 64);
                if (written[to / 64] & bit) return BCA_ERR_BAD_PAGE;
                written[to / 64] |= bit;
            }
            for (int64_t i = 0; i < n; ++i) {
                const uint32_t from = (uint32_t)pairs[2 * i];
                if (written[from / 64] >> (from % 64) & 1) return BCA_ERR_BAD_PAGE;
            }
        } else {
            std::vector<int32_t> to((size_t)n);
            for (int64_t i = 0; i < n; ++i) to[(size_t)i] = pairs[2 * i + 1];
            std::sort(to.begin(), to.end());
            if (std::adjacent_find(to.begin(), to.end()) != to.end()) return BCA_ERR_BAD_PAGE;
            for (int64_t i = 0; i < n; ++i)
                if (std::binary_search(to.begin(), to.end(), pairs[2 * i])) return BCA_ERR_BAD_PAGE;
        }
    } catch (const std::bad_alloc &) {
        return BCA_ERR_NO_MEMORY;
    }
    int rc = on_its_device(c);
    if (rc != BCA_OK) return rc;
    if (n == 0) return BCA_OK;
    if (!k_pages || !v_pages) return BCA_ERR_INVALID_ARGUMENT;
    if (!aligned(k_pages, 16) || !aligned(v_pages, 16)) return BCA_ERR_MISALIGNED;
    return bca::launch_paged_copy(c, pairs, n, k_pages, v_pages, static_cast<cudaStream_t>(stream));
}

size_t bca_paged_workspace_bytes(bca_paged_t cache, int64_t nq, int32_t slices, int32_t width) {
    if (!cache || nq <= 0 || slices <= 0 || width < 0) return 0;
    return bca::paged_workspace_bytes(cache->cache, nq, slices, width);
}

size_t bca_paged_max_workspace_bytes(bca_paged_t cache) {
    return cache ? bca::paged_max_workspace_bytes(cache->cache) : 0;
}

int bca_paged_attend(bca_paged_t cache, const void *q, int64_t nq, const int32_t *pos, const float *q_gain,
                     const void *k_pages, const void *v_pages, const int32_t *table, int32_t seqs, int32_t width,
                     const int32_t *off, const int32_t *seq, const int32_t *k_begin, const int32_t *k_end,
                     int32_t slices, int causal, void *o, float *lse, void *workspace, void *stream) {
    if (!cache || nq < 0 || seqs < 0 || width < 0 || slices < 0) return BCA_ERR_INVALID_ARGUMENT;
    const PagedCache &c = cache->cache;
    if (nq > INT32_MAX || width > INT32_MAX / bca::kPage) return BCA_ERR_INVALID_ARGUMENT;
    int rc = on_its_device(c);
    if (rc != BCA_OK) return rc;
    if (nq == 0 || slices == 0) return BCA_OK;  // (arrays of no rows may be null)
    if (q_gain && !pos) return BCA_ERR_INVALID_ARGUMENT;
    if (!q || !k_pages || !v_pages || !off || !k_begin || !k_end || !o || (seqs > 0 && width > 0 && !table))
        return BCA_ERR_INVALID_ARGUMENT;
    if (!workspace && bca::paged_workspace_bytes(c, nq, slices, width) > 0) return BCA_ERR_INVALID_ARGUMENT;
    for (const void *p : {q, k_pages, v_pages, (const void *)o, (const void *)workspace})
        if (!aligned(p, 16)) return BCA_ERR_MISALIGNED;
    for (const void *p : {(const void *)pos, (const void *)q_gain, (const void *)table, (const void *)off,
                          (const void *)seq, (const void *)k_begin, (const void *)k_end, (const void *)lse})
        if (!aligned(p, 4)) return BCA_ERR_MISALIGNED;
    return bca::launch_paged_attend(c,
                                    {q, nq, pos, q_gain, k_pages, v_pages, table, seqs, width, off, seq, k_begin,
                                     k_end, slices, causal != 0, o, lse, workspace},
                                    static_cast<cudaStream_t>(stream));
}

int bca_paged_status(bca_paged_t cache, void *stream) {
    if (!cache) return BCA_ERR_INVALID_ARGUMENT;
    const PagedCache &c = cache->cache;
    int rc = on_its_device(c);
    if (rc != BCA_OK) return rc;
    int h = 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (cudaMemcpyAsync(&h, c.d_status, sizeof(int), cudaMemcpyDeviceToHost, s) != cudaSuccess) return BCA_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return BCA_ERR_CUDA;
    // one kind of error a call; what else there is, or comes up meanwhile, is left for the next
    const struct {
        int bit, code;
    } kinds[] = {{bca::kPagedTimeout, BCA_ERR_DEVICE_TIMEOUT},
                 {bca::kPagedWorkspace, BCA_ERR_INVALID_ARGUMENT},
                 {bca::kPagedNoPage, BCA_ERR_BAD_PAGE}};
    for (const auto &k : kinds)
        if (h & k.bit) {
            if (bca::launch_paged_status_clear(c, k.bit, s) != BCA_OK) return BCA_ERR_CUDA;
            return cudaStreamSynchronize(s) == cudaSuccess ? k.code : BCA_ERR_CUDA;
        }
    return BCA_OK;
}

}  // extern "C"
