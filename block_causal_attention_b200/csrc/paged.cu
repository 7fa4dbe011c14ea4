// The paged KV cache on sm_100a: writing new tokens into pages, copying pages, and the
// launches of attention over pages (paged_rows.cu, paged_tiles.cu) with the pass that joins
// the pieces of items that several blocks shared.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "paged_device.cuh"

namespace bca {

namespace {

// ------------------------------------------------------------------ writing new tokens
//
// k_hat = R(pos) (gain * k / sqrt(mean k^2 + eps)) in fp16, v as it is, both into the layout
// of the pages.  Bound by memory: 4 D Hkv bytes read and as many written a token.  Measured on
// the device: 43,200 tokens of 8 heads, D = 48, 27.8 us, 4.8 TB/s (2.3 waves of blocks, each 50 KB on
// the way).
//
// A block takes the (up to) 32 tokens of one 32-aligned stretch of a page and up to eight KV
// heads.  Their rows come to shared memory by bulk copies, one a token, issued before anything
// else is computed: 50 KB on the way a block, four blocks a multiprocessor.  The angles (fixed
// point, sine and cosine) are computed once a token for all heads.  Keys: a warp has a head, a
// lane a token, so that the stores of a 16-byte chunk are 512 contiguous bytes.  Values: 8 x 8
// matrices turned by ldmatrix.trans; two tokens of a channel a lane, 128 contiguous bytes a
// store, and the pieces of a group of eight tokens that are not this call's are left out.
// Rows of an odd number of 16-byte units keep both from bank conflicts.

constexpr int kWriteTokens = 32;
constexpr int kWriteThreads = 256;
constexpr int kWriteHeads = 8;

struct WriteArgs {
    const void *k, *v;
    const int32_t *pos;
    const float *k_gain;
    const int32_t *table, *off, *start;
    __half *k_pages;
    void *v_pages;
    int *status;
    int64_t n, pages;
    int seqs, width, hkv;
    float eps;
    uint64_t timeout_ns;
    uint64_t turns[24];
};

// The block of 32-aligned tokens that this grid block has.  Sequence b begins at grid block
// off[b] / 32 + 2 b: tokens that need not begin at a multiple of 32 touch at most n / 32 + 2
// stretches, which is what is left before sequence b + 1.
struct WriteTile {
    int64_t row;   // of the first token
    int64_t at;    // its position in the sequence
    int count;     // tokens
    int b;
};

__device__ __forceinline__ bool write_tile(const WriteArgs &a, WriteTile &t) {
    const int64_t x = blockIdx.x;
    int before = 0;
    for (int base = 0; base < a.seqs; base += kWriteThreads) {
        const int b = base + (int)threadIdx.x;
        const bool in = b < a.seqs && min(max((int64_t)__ldg(a.off + b), (int64_t)0), a.n) / kWriteTokens + 2 * (int64_t)b <= x;
        const int c = __syncthreads_count(in);
        before += c;
        if (c < kWriteThreads) break;
    }
    if (before == 0) return false;
    t.b = before - 1;
    const int64_t o0 = min(max((int64_t)__ldg(a.off + t.b), (int64_t)0), a.n);
    const int64_t o1 = min(max((int64_t)__ldg(a.off + t.b + 1), o0), a.n);
    const int64_t s = __ldg(a.start + t.b);
    const int64_t first = ((s >> 5) + (x - (o0 / kWriteTokens + 2 * (int64_t)t.b))) * kWriteTokens;
    const int64_t lo = max(first, s), hi = min(first + kWriteTokens, s + (o1 - o0));
    if (lo >= hi) return false;
    t.at = lo;
    t.row = o0 + (lo - s);
    t.count = (int)(hi - lo);
    return true;
}

template <int D>
struct WriteSmem {
    static constexpr int STRIDE = kWriteHeads * D * 2 + 16;  // bytes of a token; 16 times an odd number
    static constexpr int OFF_V = kWriteTokens * STRIDE;
    static constexpr int OFF_TURN = 2 * OFF_V;               // cos, sin [pair][token]
    static constexpr int OFF_GAIN = OFF_TURN + D / 2 * kWriteTokens * 8;
    static constexpr int OFF_BAR = OFF_GAIN + D * 4;
    static constexpr int BYTES = OFF_BAR + 8;
};

template <int D, typename T>
__global__ void __launch_bounds__(kWriteThreads) paged_write_kernel(const __grid_constant__ WriteArgs a) {
    using L = WriteSmem<D>;
    constexpr int P = Geo<D>::PAIRS;
    constexpr int C = D / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = sm100::smem_u32(smem), bar = sbase + L::OFF_BAR;
    float2 *turn = reinterpret_cast<float2 *>(smem + L::OFF_TURN);
    float *gain = reinterpret_cast<float *>(smem + L::OFF_GAIN);
    if (threadIdx.x == 0) {
        sm100::mbar_init(bar, 1);
        sm100::mbar_fence_init();
    }
    WriteTile t;
    if (!write_tile(a, t)) return;  // its barriers are also the one behind mbar_init
    const int64_t page_at = t.at / kPage;
    int64_t page = -1;
    if (t.at >= 0 && page_at < a.width) page = __ldg(a.table + (int64_t)t.b * a.width + page_at);
    if (page < 0 || page >= a.pages) {
        if (threadIdx.x == 0) atomicOr(a.status, kPagedNoPage);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int first = (int)(t.at % kWriteTokens), slot0 = (int)(t.at % kPage) - first;  // token i of the stretch: row i
    const int h0 = blockIdx.y * kWriteHeads, heads = min(kWriteHeads, a.hkv - h0);
    const bool mine = lane >= first && lane < first + t.count;
    const int64_t row = t.row + lane - first;
    if (warp == 0) {
        const uint32_t bytes = heads * D * 2;
        if (lane == 0) sm100::mbar_arrive_expect_tx(bar, 2 * t.count * bytes);
        __syncwarp();
        if (mine) {
            const int64_t at = (row * a.hkv + h0) * D;
            sm100::bulk_g2s(sbase + lane * L::STRIDE, static_cast<const T *>(a.k) + at, bytes, bar);
            sm100::bulk_g2s(sbase + L::OFF_V + lane * L::STRIDE, static_cast<const T *>(a.v) + at, bytes, bar);
        }
    }
    if (a.pos) {
#pragma unroll 1
        for (int p = warp; p < D / 2; p += kWriteThreads / 32)
            if (mine)
                turn[p * kWriteTokens + lane] =
                    p < 3 * P ? paged_cos_sin(__ldg(a.pos + row * 3 + p / P), a.turns[8 * (p / P) + p % P])
                              : make_float2(1.f, 0.f);
        if (threadIdx.x < D) gain[threadIdx.x] = a.k_gain ? __ldg(a.k_gain + threadIdx.x) : 1.f;
        __syncthreads();
    }
    if (!sm100::mbar_wait(bar, 0, a.timeout_ns)) {
        if (threadIdx.x == 0) atomicOr(a.status, kPagedTimeout);
        sm100::mbar_wait(bar, 0, a.timeout_ns);  // the copies' memory must not be given back before they land
        return;
    }

    if (warp >= heads) return;

    // keys: twice over the row in shared memory, so that the code stays short (a call of few tokens
    // takes as long as its instructions take to come)
    if (mine) {
        const uint4 *src = reinterpret_cast<const uint4 *>(smem + lane * L::STRIDE + warp * D * 2);
        uint4 *dst = reinterpret_cast<uint4 *>(a.k_pages) + (page * a.hkv + h0 + warp) * C * kPage + slot0 + lane;
        auto chunk = [&](int c, float (&x)[8]) {
            const uint4 raw = src[c];
            const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = Io<T>::unpack(w[i]);
                x[2 * i] = f.x;
                x[2 * i + 1] = f.y;
            }
        };
        float r = 1.f;
        if (a.pos) {
            float ss[2] = {0.f, 0.f};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float x[8];
                chunk(c, x);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss[i & 1] = fmaf(x[i], x[i], ss[i & 1]);
            }
            r = rsqrtf((ss[0] + ss[1]) * (1.0f / D) + a.eps);
        }
#pragma unroll 2
        for (int c = 0; c < C; ++c) {
            float x[8];
            chunk(c, x);
            if (a.pos) {
                const float4 *gn = reinterpret_cast<const float4 *>(gain) + 2 * c;
                const float g[8] = {gn[0].x, gn[0].y, gn[0].z, gn[0].w, gn[1].x, gn[1].y, gn[1].z, gn[1].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 cs = turn[(4 * c + i) * kWriteTokens + lane];
                    const float y0 = x[2 * i] * r * g[2 * i], y1 = x[2 * i + 1] * r * g[2 * i + 1];
                    x[2 * i] = y0 * cs.x - y1 * cs.y;
                    x[2 * i + 1] = y0 * cs.y + y1 * cs.x;
                }
            }
            dst[c * kPage] = make_uint4(sm100::pack_f16x2(x[0], x[1]), sm100::pack_f16x2(x[2], x[3]),
                                        sm100::pack_f16x2(x[4], x[5]), sm100::pack_f16x2(x[6], x[7]));
        }
    }
    __syncwarp();

    // values: the four groups of eight tokens of eight channels at a time; the lane gets channel
    // lane / 4, tokens 2 (lane % 4) and the next of each
    const uint32_t from = sbase + L::OFF_V + lane * L::STRIDE + warp * D * 2;
    uint16_t *dst = static_cast<uint16_t *>(a.v_pages) +
                    (((page * a.hkv + h0 + warp) * 16 + slot0 / 8) * D + lane / 4) * 8 + 2 * (lane % 4);
    uint32_t have = 0;  // bits 2 k, 2 k + 1: the lane's two tokens of group k are this call's
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int i = 8 * k + 2 * (lane % 4) + j;
            have |= (uint32_t)(i >= first && i < first + t.count) << (2 * k + j);
        }
#pragma unroll 2
    for (int c = 0; c < C; ++c) {
        uint32_t r[4];
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(from + c * 16)
                     : "memory");
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            uint16_t *to = dst + (k * D + c * 8) * 8;
            const uint32_t both = have >> (2 * k) & 3u;
            if (both == 3u) {
                *reinterpret_cast<uint32_t *>(to) = r[k];
            } else {
                if (both & 1u) to[0] = (uint16_t)r[k];
                if (both & 2u) to[1] = (uint16_t)(r[k] >> 16);
            }
        }
    }
}

// ------------------------------------------------------------------ copying pages
//
// The page numbers travel as kernel arguments (at most 32,764 bytes of them), so the call
// needs neither a device buffer nor a copy that would have to outlive it.  Bound by memory:
// a block moves 16 KB of a page, four 16-byte loads in flight a thread.  Measured on
// the device: 805 MB in 123.5 us, 6.5 TB/s; 48 pages of 196 KB in 3.1 us.

constexpr int kCopyThreads = 256;
constexpr int kCopyUnits = 1024;  // 16-byte units a block

struct CopyArgs {
    uint4 *k_pages, *v_pages;
    int64_t page_units, pool_units;
    int parts;
};
template <int N>
struct CopyPairs {
    int2 p[N];
};

template <int N>
__global__ void __launch_bounds__(kCopyThreads) paged_copy_kernel(const __grid_constant__ CopyArgs a,
                                                                  const __grid_constant__ CopyPairs<N> pairs) {
    const int2 p = pairs.p[blockIdx.x / a.parts];
    uint4 *pool = (blockIdx.z ? a.v_pages : a.k_pages) + blockIdx.y * a.pool_units;
    const uint4 *src = pool + p.x * a.page_units;
    uint4 *dst = pool + p.y * a.page_units;
    const int64_t u0 = (int64_t)(blockIdx.x % a.parts) * kCopyUnits + threadIdx.x;
    uint4 x[kCopyUnits / kCopyThreads];
#pragma unroll
    for (int i = 0; i < kCopyUnits / kCopyThreads; ++i)
        if (u0 + i * kCopyThreads < a.page_units) x[i] = __ldcs(src + u0 + i * kCopyThreads);
#pragma unroll
    for (int i = 0; i < kCopyUnits / kCopyThreads; ++i)
        if (u0 + i * kCopyThreads < a.page_units) __stcs(dst + u0 + i * kCopyThreads, x[i]);
}

template <int N>
int launch_copy(const CopyArgs &a, const PagedCache &c, const int32_t *pairs, int64_t n, cudaStream_t stream) {
    CopyPairs<N> p;
    std::memcpy(p.p, pairs, (size_t)n * sizeof(int2));
    const dim3 grid((unsigned)(n * a.parts), (unsigned)c.layers, 2);
    paged_copy_kernel<N><<<grid, kCopyThreads, 0, stream>>>(a, p);
    return cudaGetLastError() == cudaSuccess ? BCA_OK : BCA_ERR_CUDA;
}

// ------------------------------------------------------------------ joining the pieces
//
// O = sum_p 2^(r_p - r) O_p / sum_p 2^(r_p - r) l_p with r the largest reference, over the
// pieces p of an item, always in the order of the blocks that made them.  Block c joins the
// item that share c begins and does not end.  A warp takes a row: first its pieces' references
// and sums, a lane each, then O, eight lanes a piece, with the loads of 32 pieces on the way
// at a time: three trips to memory whatever their number up to 32, and two, four rows a warp,
// for up to four.
//
// "No keys" is a sum of exactly 0: a key with a finite score adds at least its own weight, and one
// whose score is NaN leaves NaN in the sum and in O, while the reference, a running maximum, stays
// where it was, at -inf if nothing else was seen.  A piece whose sum is NaN takes part: its weight,
// 2^(-inf - r) = 0 or, beside nothing finite, NaN, times NaN is NaN in the sum and in O.

// Calls that go by clusters: 16-row tiles, few items, tables up to this wide.  Measured with one
// query token, us by clusters / by shares, D = 24 and D = 48:
//   items, tokens     1,000               8,000               16,000              32,000
//    8             5.6/9.0  5.7/10.3   8.6/10.3  9.2/11.6  12/12  13/14        18/14  20/16
//   16             6.0/9.2   11/11     9.2/12     17/14    13/15  24/17        20/20  40/23
//   32              10/10    16/12      14/15     25/17    19/20  38/24        28/32  64/41
// (At D = 48 a multiprocessor has registers for one block of a cluster, so 16 clusters do not run
// at once.  32-row tiles gain at no size: 12.3/11.1 at 8 items of 1,000 tokens.)
constexpr int kClusterPages = 96;
int cluster_items(int d) { return d == 48 ? 8 : 16; }

constexpr int kJoinThreads = 256;
constexpr int kJoinFew = 4;  // pieces that are joined in one go

template <int D, typename T>
__global__ void __launch_bounds__(kJoinThreads, 3) paged_join_kernel(const __grid_constant__ PagedArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int c = blockIdx.x;
    const PagedJoin j = a.joins[c];
    const int pieces = j.last - c + 1;
    if (j.last < c) return;
    // The workspace is the caller's.  Two calls that overlap with one workspace may read each
    // other's notes: their results are lost, but nothing outside their arrays is touched.
    if (j.last >= paged_shares(a.rows) || (uint32_t)j.g >= (uint32_t)a.hkv || (uint32_t)j.head >= (uint32_t)a.group ||
        j.left > a.rows) {
        if (threadIdx.x == 0) atomicOr(a.status, kPagedWorkspace);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / 8, e = lane % 8;
    const size_t slot = (size_t)a.rows * (D + 2);
    const int rows = a.rows / gridDim.y, row_end = min((int)(blockIdx.y + 1) * rows, j.left);
    // O / l and the LSE of a row, eight lanes
    auto write = [&](int row, float ref, float sum, const float (&o)[D / 8]) {
        const bool none = ref == -INFINITY && sum == 0.f;
        const float inv = none ? 0.f : 1.f / sum;
        const uint32_t packed = j.head + row;
        const int64_t token = (int64_t)j.row + j.token + (int32_t)(packed / a.group);
        const int head = j.g * a.group + (int)(packed % a.group);
        if ((uint64_t)token >= (uint64_t)a.nq) {
            if (e == 0) atomicOr(a.status, kPagedWorkspace);
            return;
        }
        const int64_t at = (token * a.hq + head) * D;
#pragma unroll
        for (int k = 0; k < D / 8; ++k) {
            const float y = none ? 0.f : o[k] * inv;
            if (a.o_fp32) static_cast<float *>(a.o)[at + e + 8 * k] = y;
            else static_cast<T *>(a.o)[at + e + 8 * k] = T(y);
        }
        if (a.lse && e == 0)
            a.lse[head * a.nq + token] = none ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
    };

    if (pieces <= kJoinFew) {
        // few pieces, as the 384-row tiles have: four rows a warp, everything of a row on the way at once
        for (int row = blockIdx.y * rows + 4 * warp + sub; row < row_end; row += kJoinThreads / 8) {
            float r[kJoinFew], l[kJoinFew], y[kJoinFew][D / 8];
#pragma unroll
            for (int x = 0; x < kJoinFew; ++x) {
                const float *part = a.part + (2 * (size_t)(c + x) + (x == 0 ? 1 : 0)) * slot;
                const bool on = x < pieces;
                r[x] = on ? part[(size_t)a.rows * D + row] : -INFINITY;
                l[x] = on ? part[(size_t)a.rows * (D + 1) + row] : 0.f;
#pragma unroll
                for (int k = 0; k < D / 8; ++k) y[x][k] = on ? part[(size_t)row * D + e + 8 * k] : 0.f;
            }
            float top = r[0], sum = 0.f, o[D / 8] = {};
#pragma unroll
            for (int x = 1; x < kJoinFew; ++x) top = fmaxf(top, r[x]);
#pragma unroll
            for (int x = 0; x < kJoinFew; ++x) {
                if (l[x] == 0.f) continue;  // a piece without keys: it may have no O
                const float w = sm100::ex2(r[x] - top);
                sum = fmaf(l[x], w, sum);
#pragma unroll
                for (int k = 0; k < D / 8; ++k) o[k] = fmaf(y[x][k], w, o[k]);
            }
            write(row, top, sum, o);
        }
        return;
    }

    for (int row = blockIdx.y * rows + warp; row < row_end; row += kJoinThreads / 32) {
        float ref = -INFINITY, sum = 0.f, o[D / 8] = {};
        for (int base = 0; base < pieces; base += 32) {
            const int x = base + lane;
            const float *part = a.part + (2 * (size_t)(c + x) + (x == 0 ? 1 : 0)) * slot;
            float r = -INFINITY, l = 0.f;
            if (x < pieces) {
                r = part[(size_t)a.rows * D + row];
                l = part[(size_t)a.rows * (D + 1) + row];
            }
            float top = r;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
            top = fmaxf(top, ref);
            const bool some = l != 0.f;  // else a piece without keys: it may have no O
            if (!__any_sync(0xffffffffu, some)) continue;
            const float keep = ref == -INFINITY ? 0.f : sm100::ex2(ref - top);
            const float w = some ? sm100::ex2(r - top) : 0.f;
            if (some) l *= w;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) l += __shfl_xor_sync(0xffffffffu, l, s);
            sum = sum * keep + l;
            ref = top;
            float y[8][D / 8];
            const float *first = a.part + (size_t)row * D + e;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int z = base + 4 * i + sub;
                const bool on = __shfl_sync(0xffffffffu, some, 4 * i + sub);
                const float *from = first + (2 * (size_t)(c + z) + (z == 0 ? 1 : 0)) * slot;
#pragma unroll
                for (int k = 0; k < D / 8; ++k) y[i][k] = on ? from[8 * k] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < D / 8; ++k) o[k] *= keep;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float m = __shfl_sync(0xffffffffu, w, 4 * i + sub);
#pragma unroll
                for (int k = 0; k < D / 8; ++k) o[k] = fmaf(y[i][k], m, o[k]);
            }
        }
#pragma unroll
        for (int s = 8; s < 32; s <<= 1)
#pragma unroll
            for (int k = 0; k < D / 8; ++k) o[k] += __shfl_xor_sync(0xffffffffu, o[k], s);
        if (sub == 0) write(row, ref, sum, o);
        __syncwarp();
    }
}

template <int D, typename T>
int launch_join(const PagedArgs &a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)paged_shares(a.rows), (unsigned)(a.rows <= 32 ? a.rows / 8 : a.rows / 32));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_join_kernel<D, T>, a) == cudaSuccess ? BCA_OK : BCA_ERR_CUDA;
}

// ------------------------------------------------------------------ the status word

// Takes one reported bit back.  Kernels of other streams may set bits at any time, so the word is
// never written as a whole.
__global__ void paged_status_clear_kernel(int *status, int bit) { atomicAnd(status, ~bit); }

// ------------------------------------------------------------------ by head size and type

template <typename F>
int by_type(const PagedCache &c, F &&f) {
    const bool f16 = (c.flags & BCA_PAGED_FP16) != 0;
    switch (c.d) {
        case 24: return f16 ? f(std::integral_constant<int, 24>{}, __half{}) : f(std::integral_constant<int, 24>{}, __nv_bfloat16{});
        case 32: return f16 ? f(std::integral_constant<int, 32>{}, __half{}) : f(std::integral_constant<int, 32>{}, __nv_bfloat16{});
        case 48: return f16 ? f(std::integral_constant<int, 48>{}, __half{}) : f(std::integral_constant<int, 48>{}, __nv_bfloat16{});
        default: return BCA_ERR_UNSUPPORTED;
    }
}

}  // namespace

// Tiles of 16, 32, 128 or 384 packed rows, by the rows of an average slice (the sizes of single
// ones are device data).  Measured on 16 sequences of 8,000 tokens and 8 KV heads and on one of
// 20,000, D = 24 / 48, us:
//   rows of a slice       16         32         64         128        256        512       1 x 64    1 x 384
//   16-row tiles        32 / 39    57 / 68   109 / 123  212 / 237  416 / 464  826 / 927   26 / 30  102 / 110
//   32-row tiles        39 / 45    40 / 47    73 / 82   138 / 152  266 / 290  523 / 571   20 / 23   65 / 70
//   128-row tiles       68 / 78    69 / 80    69 / 81    71 / 83   121 / 136  222 / 253   33 / 41   47 / 57
//   384-row tiles       90 / 110   90 / 111   90 / 112   92 / 114  121 / 154  227 / 286   36 / 45   52 / 72
// and on chunks, 128- against 384-row tiles: the 4.5B window 1,016 / 876 us, half a 720p chunk
// 2,270 / 2,220, ragged chunks of several streams 408 / 322.
// All of these are slices of like sizes.  A call that mixes sizes gets the average's tiles for all:
// 31 single tokens over 1,000 to 31,000 keys beside a chunk of 2,001 over 5,000 (128 heads of 8,
// D = 48) take 1,011 us in one call, 140 and 673 in two; 1,023 single tokens over 100 to 1,100 keys
// beside a chunk of 300 over 8,000 take 1,562, against 463 and 150.  Two calls are the way there.
PagedShape paged_shape(const PagedCache &c, int64_t nq, int slices, int width) {
    const int64_t group = c.hq / c.hkv, rows = nq * group / std::max(slices, 1);
    PagedShape s = {rows <= 16 ? 16 : rows <= 64 ? 32 : rows <= 256 ? kPagedNarrowRows : kPagedTileRows, 0};
    if (s.rows == 16 && nq <= 1024 && slices <= 1024) {
        const int64_t items = (nq * group + (int64_t)slices * (s.rows - 1)) / s.rows * c.hkv;
        if (items <= cluster_items(c.d) && width <= kClusterPages) s.items = (int)items;
    }
    return s;
}

static size_t shares_bytes(const PagedCache &c, int rows) {
    return paged_shares(rows) * (kPagedJoinBytes + 2 * (size_t)rows * (c.d + 2) * sizeof(float));
}

size_t paged_workspace_bytes(const PagedCache &c, int64_t nq, int slices, int width) {
    const PagedShape s = paged_shape(c, nq, slices, width);
    return s.items > 0 ? 0 : shares_bytes(c, s.rows);
}

size_t paged_max_workspace_bytes(const PagedCache &c) {
    size_t most = 0;
    for (int rows : {16, 32, kPagedNarrowRows, kPagedTileRows}) most = std::max(most, shares_bytes(c, rows));
    return most;
}

int prepare_paged(const PagedCache &c) {
    int rc = by_type(c, [](auto d, auto t) {
        using L = WriteSmem<decltype(d)::value>;
        return cudaFuncSetAttribute(paged_write_kernel<decltype(d)::value, decltype(t)>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, L::BYTES) == cudaSuccess
                   ? BCA_OK
                   : BCA_ERR_CUDA;
    });
    if (rc != BCA_OK) return rc;
    rc = prepare_paged_rows(c);
    return rc == BCA_OK ? prepare_paged_tiles(c) : rc;
}

int launch_paged_write(const PagedCache &c, const PagedWriteIO &io, cudaStream_t stream) {
    WriteArgs a;
    a.k = io.k;
    a.v = io.v;
    a.pos = io.pos;
    a.k_gain = io.k_gain;
    a.table = io.table;
    a.off = io.off;
    a.start = io.start;
    a.k_pages = static_cast<__half *>(io.k_pages);
    a.v_pages = io.v_pages;
    a.status = c.d_status;
    a.n = io.n;
    a.pages = c.pages;
    a.seqs = io.seqs;
    a.width = io.width;
    a.hkv = c.hkv;
    a.eps = c.eps;
    a.timeout_ns = kPagedWaitNs;
    std::memcpy(a.turns, c.turns, sizeof(a.turns));
    const int64_t blocks = io.n / kWriteTokens + 2 * (int64_t)io.seqs;
    if (blocks > INT32_MAX) return BCA_ERR_TOO_LARGE;
    return by_type(c, [&](auto d, auto t) {
        const dim3 grid((unsigned)blocks, (unsigned)((c.hkv + kWriteHeads - 1) / kWriteHeads));
        paged_write_kernel<decltype(d)::value, decltype(t)>
            <<<grid, kWriteThreads, WriteSmem<decltype(d)::value>::BYTES, stream>>>(a);
        return cudaGetLastError() == cudaSuccess ? BCA_OK : BCA_ERR_CUDA;
    });
}

int launch_paged_copy(const PagedCache &c, const int32_t *pairs, int64_t n, void *k_pages, void *v_pages,
                      cudaStream_t stream) {
    CopyArgs a;
    a.k_pages = static_cast<uint4 *>(k_pages);
    a.v_pages = static_cast<uint4 *>(v_pages);
    a.page_units = (int64_t)c.hkv * c.d * kPage / 8;
    a.pool_units = a.page_units * c.pages;
    const int64_t parts = (a.page_units + kCopyUnits - 1) / kCopyUnits;
    if (parts > INT32_MAX / 4000) return BCA_ERR_TOO_LARGE;
    a.parts = (int)parts;
    // A launch's arguments are copied whatever part of them is used, hence two sizes.
    for (int64_t at = 0; at < n;) {
        const int64_t m = std::min<int64_t>(n - at, n - at <= 480 ? 480 : 4000);
        const int rc = m <= 480 ? launch_copy<480>(a, c, pairs + 2 * at, m, stream)
                                : launch_copy<4000>(a, c, pairs + 2 * at, m, stream);
        if (rc != BCA_OK) return rc;
        at += m;
    }
    return BCA_OK;
}

int launch_paged_status_clear(const PagedCache &c, int bit, cudaStream_t stream) {
    paged_status_clear_kernel<<<1, 1, 0, stream>>>(c.d_status, bit);
    return cudaGetLastError() == cudaSuccess ? BCA_OK : BCA_ERR_CUDA;
}

int launch_paged_attend(const PagedCache &c, const PagedAttendIO &io, cudaStream_t stream) {
    const PagedShape s = paged_shape(c, io.nq, io.slices, io.width);
    PagedArgs a;
    a.q = io.q;
    a.pos = io.pos;
    a.q_gain = io.q_gain;
    a.k_pages = io.k_pages;
    a.v_pages = io.v_pages;
    a.table = io.table;
    a.off = io.off;
    a.seq = io.seq;
    a.k_begin = io.k_begin;
    a.k_end = io.k_end;
    a.o = io.o;
    a.lse = io.lse;
    a.joins = static_cast<PagedJoin *>(io.workspace);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(io.workspace) + (size_t)paged_shares(s.rows) * kPagedJoinBytes);
    a.status = c.d_status;
    a.nq = io.nq;
    a.pages = c.pages;
    a.seqs = io.seqs;
    a.width = io.width;
    a.slices = io.slices;
    a.causal = io.causal;
    a.hq = c.hq;
    a.hkv = c.hkv;
    a.group = c.hq / c.hkv;
    a.rows = s.rows;
    a.o_fp32 = (c.flags & BCA_O_FP32) ? 1 : 0;
    a.eps = c.eps;
    a.scale = 1.4426950408889634f / std::sqrt((float)c.d);
    a.timeout_ns = (c.flags & BCA_TEST_FORCE_TIMEOUT) ? 1000000ull : kPagedWaitNs;
    a.skip_loads = (c.flags & BCA_TEST_FORCE_TIMEOUT) ? 1 : 0;
    std::memcpy(a.turns, c.turns, sizeof(a.turns));
    // The row of items, at its longest: see paged_device.cuh.
    const double items = ((double)io.nq * a.group / a.rows + io.slices) * c.hkv;
    const double keys = std::max((double)io.width * kPage, (double)io.nq);
    a.shift = 0;
    while (a.shift < 27 && items * (64.0 + std::ldexp(keys, -4 - a.shift)) > 2e9) ++a.shift;
    if (items * 65.0 > 2e9) return BCA_ERR_TOO_LARGE;
    const int rc =
        a.rows >= kPagedNarrowRows ? launch_paged_tiles(c, a, stream) : launch_paged_rows(c, a, s.items, stream);
    if (rc != BCA_OK || s.items > 0) return rc;
    return by_type(c, [&](auto d, auto t) { return launch_join<decltype(d)::value, decltype(t)>(a, stream); });
}

}  // namespace bca
