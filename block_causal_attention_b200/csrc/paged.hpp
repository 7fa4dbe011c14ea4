// Paged KV cache: the host handle and the launch interface between the C ABI
// (paged_api.cpp) and the CUDA kernels.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/bca.h"

namespace bca {

constexpr int kPage = BCA_PAGE_TOKENS;
constexpr int kPagedJoinBytes = 32;  // of the workspace, for each share
constexpr int kPagedTileRows = 384;  // packed rows of a work item of paged_tiles.cu
constexpr int kPagedNarrowRows = 128;  // and of its form for slices of few
// Blocks of an attention call with tiles of so many rows: all that run at once.
constexpr int paged_shares(int rows) { return rows == kPagedNarrowRows ? 296 : 148; }

// status-word bits written by the paged kernels
constexpr int kPagedTimeout = 0x1;
constexpr int kPagedNoPage = 0x2;
constexpr int kPagedWorkspace = 0x4;

struct PagedCache {
    int hq = 0, hkv = 0, d = 0, layers = 1;
    int64_t pages = 0;
    float eps = 1e-6f;
    uint32_t flags = 0;
    // turns per unit of position of pair i of axis a: base_a^(-i/P) / 2 pi without the whole
    // ones, in units of 2^-64, at [8 a + i]
    uint64_t turns[24] = {};
    int device = -1;
    int *d_status = nullptr;
};

struct PagedWriteIO {
    const void *k, *v;
    int64_t n;
    const int32_t *pos;
    const float *k_gain;
    const int32_t *table;
    int seqs, width;
    const int32_t *off, *start;
    void *k_pages, *v_pages;
};

struct PagedAttendIO {
    const void *q;
    int64_t nq;
    const int32_t *pos;
    const float *q_gain;
    const void *k_pages, *v_pages;
    const int32_t *table;
    int seqs, width;
    const int32_t *off, *seq, *k_begin, *k_end;
    int slices;
    int causal;
    void *o;
    float *lse;
    void *workspace;
};

// How a call of these sizes is cut (the same for the workspace and the launch): tiles of `rows`
// packed (token, head of the KV group) rows; items > 0: that many (tile, KV head) items, a cluster
// of blocks each; 0: equal shares of whatever there is.
struct PagedShape {
    int rows;
    int items;
};
PagedShape paged_shape(const PagedCache &c, int64_t nq, int slices, int width);
size_t paged_workspace_bytes(const PagedCache &c, int64_t nq, int slices, int width);
size_t paged_max_workspace_bytes(const PagedCache &c);  // of any sizes

int prepare_paged(const PagedCache &c);
int launch_paged_write(const PagedCache &c, const PagedWriteIO &io, cudaStream_t stream);
int launch_paged_copy(const PagedCache &c, const int32_t *pairs, int64_t n, void *k_pages, void *v_pages,
                      cudaStream_t stream);
int launch_paged_attend(const PagedCache &c, const PagedAttendIO &io, cudaStream_t stream);
int launch_paged_status_clear(const PagedCache &c, int bit, cudaStream_t stream);

struct PagedArgs;
int prepare_paged_rows(const PagedCache &c);
int launch_paged_rows(const PagedCache &c, const PagedArgs &a, int items, cudaStream_t stream);
int prepare_paged_tiles(const PagedCache &c);
int launch_paged_tiles(const PagedCache &c, const PagedArgs &a, cudaStream_t stream);

}  // namespace bca

// The opaque handle behind bca_paged_t.
struct bca_paged_s {
    bca::PagedCache cache;
};
