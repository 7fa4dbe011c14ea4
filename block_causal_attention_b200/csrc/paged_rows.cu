// Attention of few packed rows (single tokens, proposed tokens, small groups) over the pages
// of a KV cache.
//
// O_i = sum_j 2^(s_ij - r_i) v_j / sum_j 2^(s_ij - r_i), s_ij = log2(e)/sqrt(D) q_i . k_j, in
// one pass over the keys: the reference r_i follows the running maximum.
//
// Bound by memory: a key and value of a KV head are 4 D bytes for 4 D * rows operations, so at
// 16 or 32 rows even the warps' own matrix instructions keep up.  What counts is bytes in
// flight: one block a multiprocessor, a ring of whole pages (a page's keys and values of one
// head are two contiguous stretches, moved by two bulk copies) filled by one warp that runs
// ahead over page and item borders.  Eight warps take 16 of a page's 128 tokens each; their
// results meet once an item, so that one page is enough work for all of them.  Measured on the
// device: one token of 128 heads over 172,800 keys of 8 KV heads, D = 48, 49 us (5.4 TB/s with the
// launch and the joining pass, about 8 us); 32 tokens over 512,000 keys 142 us, 5.7 TB/s.
//
// The layout of the pages is that of the 8 x 8 matrices that ldmatrix reads: 8 tokens x 8
// channels of K and 8 channels x 8 tokens of V lie in 128 contiguous bytes, so both operands
// come to the registers without bank conflicts and without a transposition.
#include <cuda_runtime.h>

#include <type_traits>

#include "paged_device.cuh"
#include "paged_mma.cuh"

namespace bca {

using namespace sm100;

namespace {

constexpr int kWarps = 8;                     // consumers; one more fills the ring
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kWarpTokens = kPage / kWarps;   // 16

// LO: fp16 values; the rounding of queries made here is kept as a second fp16 tile (paged_tiles.cu has
// the reason).  Given post-prologue they take no time for it (24.7 us both ways, 64 rows); made here
// they take 26.8 us against 24.8.
template <int D, int MT, int CL, bool LO>
struct RowsSmem {
    static constexpr int TILE = D * kPage * 2;
    // one block a multiprocessor with all of its shared memory; of a cluster's blocks two (D < 48)
    static constexpr int STAGES = CL == 1 ? (D == 48 ? 7 : D == 32 ? 10 : 13) : (D == 48 ? 3 : D == 32 ? 5 : 6);
    static constexpr int QSTRIDE = D == 24 ? 40 : D + 8;  // elements; an odd number of 16-byte units
    static constexpr int OFF_RING = 0;
    static constexpr int OFF_Q = STAGES * 2 * TILE;
    static constexpr int Q_BYTES = 16 * MT * QSTRIDE * 2;
    static constexpr int OFF_MERGE = OFF_Q + (LO ? 2 : 1) * Q_BYTES;
    static constexpr int OFF_PART = OFF_MERGE + kWarps * 16 * (D + 2) * 4;  // the block's, for its cluster
    static constexpr int OFF_BAR = OFF_PART + (CL == 1 ? 0 : 16 * MT * (D + 2) * 4);
    static constexpr int OFF_HERE = OFF_BAR + 2 * (STAGES + kItemRing) * 8;
    static constexpr int OFF_ITEMS = OFF_HERE + STAGES * 4;
    static constexpr int OFF_ABORT = OFF_ITEMS + kItemRing * (int)sizeof(PagedItem);
    static constexpr int BYTES = OFF_ABORT + 4;
};

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// The same, and whether all of them said yes.
__device__ __forceinline__ bool consumers_all(bool yes) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, 256, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"((uint32_t)yes)
        : "memory");
    return all != 0;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A word of the shared memory of the cluster's block `rank`, at this block's address of it.
__device__ __forceinline__ float cluster_load(uint32_t addr, int rank) {
    uint32_t there;
    float x;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(addr), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(there) : "memory");
    return x;
}

// MT: 16-row matrix tiles a work tile has (rows = 16 MT).  CL: blocks that share an item as a
// cluster; 1: the blocks take equal shares of all items.
template <int D, typename T, int MT, int CL>
__global__ void __launch_bounds__(kThreads, 1) paged_rows_kernel(const __grid_constant__ PagedArgs a) {
    using L = RowsSmem<D, MT, CL, Io<T>::kF16>;
    constexpr int S = L::STAGES;
    constexpr int R = 16 * MT;
    constexpr int KS = D / 16;            // 16-channel steps; D = 24 has an 8-channel one behind
    constexpr bool TAIL = D % 16 != 0;
    constexpr int NV = D / 8;
    constexpr float kShift = Io<T>::kShift;

    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    volatile int *here = reinterpret_cast<volatile int *>(smem + L::OFF_HERE);
    auto full = [&](int i) -> uint32_t { return sbase + L::OFF_BAR + 8u * (uint32_t)i; };
    const uint32_t item_bars = sbase + L::OFF_BAR + 8u * (2 * S);
    PagedItem *items = reinterpret_cast<PagedItem *>(smem + L::OFF_ITEMS);
    auto empty = [&](int i) -> uint32_t { return sbase + L::OFF_BAR + 8u * (uint32_t)(S + i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // the joining kernel may be put in place as blocks of this one end
    if constexpr (CL == 1) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < S; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), kWarps);
        }
        for (int i = 0; i < kItemRing; ++i) {
            mbar_init(item_bars + 8u * i, 1);
            mbar_init(item_bars + 8u * (kItemRing + i), kWarps);
        }
        mbar_fence_init();
    }
    const int c = blockIdx.x;
    __syncthreads();

    if (warp == kWarps) {
        paged_fill<R, S, L::TILE, L::TILE, 2 * L::TILE, CL>(a, c, sbase + L::OFF_RING, full(0), item_bars, items,
                                                     here, abort_flag);
        return;
    }

    // ---------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3;
    __half *qs = reinterpret_cast<__half *>(smem + L::OFF_Q);
    float *merge = reinterpret_cast<float *>(smem + L::OFF_MERGE);
    // ldmatrix addresses inside a tile: lanes 8 j .. 8 j + 7 give the rows of matrix j.  K: chunk
    // j % 2, token group j / 2 of this warp; V: token group j % 2, channel group j / 2.
    const uint32_t kaddr = (lane >> 3 & 1) * (kPage * 16) + (2 * warp + (lane >> 4)) * 128 + (lane & 7) * 16;
    const uint32_t vaddr = ((2 * warp + (lane >> 3 & 1)) * D + 8 * (lane >> 4) + (lane & 7)) * 16;
    float2 gain[Row8<D>::N];
    Row8<D>::load_gain(a.q_gain, lane & 7, gain);
    // O / l and the LSE of row r of an item: channels e, e + 16, .. of 16 lanes
    auto write = [&](const PagedItem &x, int r, int e, float top, float l, const float (&y)[(D + 15) / 16]) {
        const bool none = top == -INFINITY && l == 0.f;  // a row whose scores are all NaN has a sum that is NaN
        const float inv = none ? 0.f : 1.f / l;
        const uint32_t packed = x.head + r;
        const int64_t token = x.row + x.token + (int32_t)(packed / a.group);
        const int head = x.g * a.group + (int)(packed % a.group);
        const int64_t at = (token * a.hq + head) * D;
#pragma unroll
        for (int i = 0; i < (D + 15) / 16; ++i) {
            if (e + 16 * i >= D) continue;
            const float z = none ? 0.f : y[i] * inv;
            if (a.o_fp32) static_cast<float *>(a.o)[at + e + 16 * i] = z;
            else static_cast<T *>(a.o)[at + e + 16 * i] = T(z);
        }
        if (a.lse && e == 0) a.lse[head * a.nq + token] = none ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
    };
    PagedItem mine;    // of a cluster
    bool has = false;
    bool ok = true;
    int it = 0;
    for (int n_item = 0;; ++n_item) {
        // A wait that ran out ends the block here, for all warps alike: they meet in barriers below.
        const int slot = n_item % kItemRing;
        if (ok) ok = paged_wait(item_bars + 8u * slot, (n_item / kItemRing) & 1, a, abort_flag);
        if (!consumers_all(ok)) break;
        const PagedItem &x = items[slot];
        const int32_t p0 = x.p0, p1 = x.p1, kb = x.kb;
        if (p0 < 0) break;

        // queries: QK-Norm and RoPE, fp16 (|q_hat| <= sqrt(D) max|gain|; 11 bits of significand
        // against bf16's 8), with what the rounding left where values are fp16.  The
        // softmax scale is applied to the scores in fp32 instead, so that bf16 queries given
        // post-prologue stay exact in fp16's normal range (below 2^-14 their last bits go, below
        // 2^-25 all of them).
        for (int r = threadIdx.x >> 3; r < R; r += kWarps * 4) {
            const int e = lane & 7;
            const bool live = r < x.left;  // the same for the eight lanes of a row
            const uint32_t packed = x.head + (live ? r : 0);
            const int64_t row = x.row + x.token + (int32_t)(packed / a.group);
            Row8<D> q;
            q.load(static_cast<const T *>(a.q) + (row * a.hq + x.g * a.group + packed % a.group) * D,
                   a.pos ? a.pos + row * 3 : static_cast<const int32_t *>(a.q), e);
            if (a.pos) q.prologue(gain, a.turns, a.eps, e);
#pragma unroll
            for (int i = 0; i < Row8<D>::N; ++i)
                if (e + 8 * i < D / 2) {
                    __half *at = qs + r * L::QSTRIDE + 2 * (e + 8 * i);
                    const float2 y = live ? q.x[i] : float2{0.f, 0.f};
                    const uint32_t hi = pack_f16x2(y.x, y.y);
                    *reinterpret_cast<uint32_t *>(at) = hi;
                    if (Io<T>::kF16 && a.pos) {
                        const float2 back = Io<__half>::unpack(hi);
                        *reinterpret_cast<uint32_t *>(at + L::Q_BYTES / 2) = pack_f16x2(y.x - back.x, y.y - back.y);
                    }
                }
        }
        consumers_sync();
        uint32_t qa[MT][KS][4], qt[MT][2];
        int32_t lim[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const __half *q0 = qs + (16 * m + g) * L::QSTRIDE + 2 * t, *q1 = q0 + 8 * L::QSTRIDE;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                qa[m][k][0] = *reinterpret_cast<const uint32_t *>(q0 + 16 * k);
                qa[m][k][1] = *reinterpret_cast<const uint32_t *>(q1 + 16 * k);
                qa[m][k][2] = *reinterpret_cast<const uint32_t *>(q0 + 16 * k + 8);
                qa[m][k][3] = *reinterpret_cast<const uint32_t *>(q1 + 16 * k + 8);
            }
            qt[m][0] = TAIL ? *reinterpret_cast<const uint32_t *>(q0 + 16 * KS) : 0u;
            qt[m][1] = TAIL ? *reinterpret_cast<const uint32_t *>(q1 + 16 * KS) : 0u;
#pragma unroll
            for (int h = 0; h < 2; ++h) lim[m][h] = x.limit(16 * m + g + 8 * h, a.group);
        }
        // keys that every row of the tile sees end here, and those that any row sees there
        const int32_t lim_all = x.limit(0, a.group), lim_any = x.limit(x.left - 1, a.group);

        float o[MT][NV][4], ref[MT][2], sum[MT][2];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int n = 0; n < NV; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) o[m][n][j] = 0.f;
            ref[m][0] = ref[m][1] = -INFINITY;
            sum[m][0] = sum[m][1] = 0.f;
        }

        for (int32_t p = p0; p < p1; ++p, ++it) {
            const int st = it % S;
            if (ok) ok = __all_sync(0xffffffffu, paged_wait(full(st), (it / S) & 1, a, abort_flag));
            if (!ok) break;
            const int32_t key0 = p * kPage + warp * kWarpTokens;
            if (here[st] && key0 + kWarpTokens > kb && key0 < lim_any) {
                const uint32_t ks = sbase + L::OFF_RING + st * 2 * L::TILE, vs = ks + L::TILE;
                uint32_t kf[KS][4], kt[2] = {0, 0}, vf[NV][2];
#pragma unroll
                for (int k = 0; k < KS; ++k) ldsm4(ks + kaddr + k * (2 * kPage * 16), kf[k]);
                if constexpr (TAIL)
                    ldsm2(ks + KS * (2 * kPage * 16) + (2 * warp + (lane >> 3 & 1)) * 128 + (lane & 7) * 16, kt[0], kt[1]);
                ldsm_v<NV>(vs + vaddr, vf);

                const bool inside = key0 >= kb && key0 + kWarpTokens <= lim_all;
                bool odd = false;  // values that are not finite, at keys that some rows do not see
                if (!inside) odd = clear_unseen<T, NV>(vf, key0 + 2 * t, kb, lim_any);
                // each step for all row tiles before the next one: their chains run side by side
                float s[MT][2][4] = {}, mx[MT][2];
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma16<true>(s[m][0], qa[m][k], kf[k][0], kf[k][1]);
                        mma16<true>(s[m][1], qa[m][k], kf[k][2], kf[k][3]);
                    }
                if constexpr (TAIL) {
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma8_f16(s[m][0], qt[m][0], qt[m][1], kt[0]);
                        mma8_f16(s[m][1], qt[m][0], qt[m][1], kt[1]);
                    }
                }
                if (Io<T>::kF16 && a.pos) {
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        const __half *q0 = qs + L::Q_BYTES / 2 + (16 * m + g) * L::QSTRIDE + 2 * t;
                        auto word = [&](int at) { return *reinterpret_cast<const uint32_t *>(q0 + at); };
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            const uint32_t lo[4] = {word(16 * k), word(8 * L::QSTRIDE + 16 * k), word(16 * k + 8),
                                                    word(8 * L::QSTRIDE + 16 * k + 8)};
                            mma16<true>(s[m][0], lo, kf[k][0], kf[k][1]);
                            mma16<true>(s[m][1], lo, kf[k][2], kf[k][3]);
                        }
                        if constexpr (TAIL) {
                            mma8_f16(s[m][0], word(16 * KS), word(8 * L::QSTRIDE + 16 * KS), kt[0]);
                            mma8_f16(s[m][1], word(16 * KS), word(8 * L::QSTRIDE + 16 * KS), kt[1]);
                        }
                    }
                }
                if (!inside) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int32_t key = key0 + 8 * n + 2 * t + (j & 1);
                                if (key < kb || key >= lim[m][j >> 1]) s[m][n][j] = -INFINITY;
                            }
                }
                bool grow = false;
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        mx[m][h] = fmaxf(fmaxf(s[m][0][2 * h], s[m][0][2 * h + 1]),
                                         fmaxf(s[m][1][2 * h], s[m][1][2 * h + 1])) * a.scale;
                        grow |= mx[m][h] > ref[m][h] + (kShift + kLazy);
                    }
                if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float top = mx[m][h];
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                            if (top > ref[m][h] + (kShift + kLazy)) {
                                const float now = top - kShift;
                                const float mul = ref[m][h] == -INFINITY ? 0.f : ex2(ref[m][h] - now);
                                ref[m][h] = now;
                                sum[m][h] *= mul;
#pragma unroll
                                for (int n = 0; n < NV; ++n) {
                                    o[m][n][2 * h] *= mul;
                                    o[m][n][2 * h + 1] *= mul;
                                }
                            }
                        }
                }
                uint32_t pa[MT][4];  // P in the values' type: it is a factor of the matrix product
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float neg = ref[m][h] == -INFINITY ? 0.f : -ref[m][h];
#pragma unroll
                        for (int n = 0; n < 2; ++n) {
                            const float y0 = ex2(fmaf(s[m][n][2 * h], a.scale, neg));
                            const float y1 = ex2(fmaf(s[m][n][2 * h + 1], a.scale, neg));
                            sum[m][h] += y0 + y1;
                            pa[m][2 * n + h] = Io<T>::pack(y0, y1);
                        }
                    }
#pragma unroll
                for (int n = 0; n < NV; ++n)
#pragma unroll
                    for (int m = 0; m < MT; ++m) mma16<Io<T>::kF16>(o[m][n], pa[m], vf[n][0], vf[n][1]);
                if (odd) {
#pragma unroll
                    for (int m = 0; m < MT; ++m)
                        add_left_out<D, T, NV>(o[m], pa[m],
                                               reinterpret_cast<const T *>(smem + (vs - sbase)) + 2 * warp * D * 8, key0,
                                               kb, lim[m]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(st));
        }

        // ------------------------------------------------ the eight warps' results meet
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float *own = merge + warp * 16 * (D + 2);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float l = sum[m][h];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                float *row = own + (g + 8 * h) * (D + 2);
#pragma unroll
                for (int n = 0; n < NV; ++n)
                    *reinterpret_cast<float2 *>(row + 8 * n + 2 * t) = make_float2(o[m][n][2 * h], o[m][n][2 * h + 1]);
                if (t == 0) {
                    row[D] = ref[m][h];
                    row[D + 1] = l;
                }
            }
            consumers_sync();
            const int r = threadIdx.x >> 4, e = threadIdx.x & 15;
            const float *row = merge + r * (D + 2);
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, row[w * 16 * (D + 2) + D]);
            float l = 0.f, y[(D + 15) / 16] = {};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float *in = row + w * 16 * (D + 2);
                const float mul = top == -INFINITY ? 0.f : ex2(in[D] - top);
                l = fmaf(in[D + 1], mul, l);
#pragma unroll
                for (int i = 0; i < (D + 15) / 16; ++i)
                    if (e + 16 * i < D) y[i] = fmaf(in[e + 16 * i], mul, y[i]);
            }
            if constexpr (CL > 1) {
                float *part = reinterpret_cast<float *>(smem + L::OFF_PART) + (16 * m + r) * (D + 2);
#pragma unroll
                for (int i = 0; i < (D + 15) / 16; ++i)
                    if (e + 16 * i < D) part[e + 16 * i] = y[i];
                if (e == 0) {
                    part[D] = top;
                    part[D + 1] = l;
                }
            } else if (16 * m + r < x.left) {
                if (x.whole) {
                    write(x, 16 * m + r, e, top, l, y);
                } else {  // without pages too: the sum, 0, tells
                    float *part = paged_part(a, D, x.part);
#pragma unroll
                    for (int i = 0; i < (D + 15) / 16; ++i)
                        if (e + 16 * i < D) part[(16 * m + r) * D + e + 16 * i] = y[i];
                    if (e == 0) {
                        part[R * D + 16 * m + r] = top;
                        part[R * (D + 1) + 16 * m + r] = l;
                    }
                }
            }
            consumers_sync();
        }
        if constexpr (CL > 1) {
            has = true;
            mine = x;
        }
        if (lane == 0) mbar_arrive(item_bars + 8u * (kItemRing + slot));
    }
    if constexpr (CL > 1) {
        // Every block comes through both barriers, also one that had nothing to do or gave up: the
        // others read its memory in between.
        __syncwarp();
        cluster_sync();
        if (has) {
            const int r = c % CL * (R / CL) + (threadIdx.x >> 4), e = threadIdx.x & 15;
            if (threadIdx.x < 16 * (R / CL) && r < mine.left) {
                const uint32_t part = sbase + L::OFF_PART + r * (D + 2) * 4;
                float ref[CL], l[CL], in[CL][(D + 15) / 16];
#pragma unroll
                for (int k = 0; k < CL; ++k) {
                    ref[k] = cluster_load(part + D * 4, k);
                    l[k] = cluster_load(part + (D + 1) * 4, k);
#pragma unroll
                    for (int i = 0; i < (D + 15) / 16; ++i)
                        in[k][i] = cluster_load(part + min(e + 16 * i, D - 1) * 4, k);
                }
                float top = ref[0], sum = 0.f, y[(D + 15) / 16] = {};
#pragma unroll
                for (int k = 1; k < CL; ++k) top = fmaxf(top, ref[k]);
#pragma unroll
                for (int k = 0; k < CL; ++k) {
                    const float mul = top == -INFINITY ? 0.f : ex2(ref[k] - top);
                    sum = fmaf(l[k], mul, sum);
#pragma unroll
                    for (int i = 0; i < (D + 15) / 16; ++i) y[i] = fmaf(in[k][i], mul, y[i]);
                }
                write(mine, r, e, top, sum, y);
            }
        }
        __syncwarp();
        cluster_sync();
    }
}

template <int D, typename T>
const void *rows_kernel(int rows, bool cluster) {
    if (cluster) return (const void *)paged_rows_kernel<D, T, 1, kCluster>;
    return rows == 16 ? (const void *)paged_rows_kernel<D, T, 1, 1> : (const void *)paged_rows_kernel<D, T, 2, 1>;
}

template <int D, typename T>
int rows_bytes(int rows, bool cluster) {
    constexpr bool LO = Io<T>::kF16;
    return cluster      ? RowsSmem<D, 1, kCluster, LO>::BYTES
           : rows == 16 ? RowsSmem<D, 1, 1, LO>::BYTES
                        : RowsSmem<D, 2, 1, LO>::BYTES;
}

template <int D>
const void *rows_kernel(bool f16, int rows, bool cluster, int &bytes) {
    bytes = f16 ? rows_bytes<D, __half>(rows, cluster) : rows_bytes<D, __nv_bfloat16>(rows, cluster);
    return f16 ? rows_kernel<D, __half>(rows, cluster) : rows_kernel<D, __nv_bfloat16>(rows, cluster);
}

const void *rows_kernel(const PagedCache &c, int rows, bool cluster, int &bytes) {
    const bool f16 = (c.flags & BCA_PAGED_FP16) != 0;
    switch (c.d) {
        case 24: return rows_kernel<24>(f16, rows, cluster, bytes);
        case 32: return rows_kernel<32>(f16, rows, cluster, bytes);
        default: return rows_kernel<48>(f16, rows, cluster, bytes);
    }
}

}  // namespace

int prepare_paged_rows(const PagedCache &c) {
    for (int rows : {16, 32})
        for (bool cluster : {false, true}) {
            if (cluster && rows != 16) continue;
            int bytes = 0;
            const void *f = rows_kernel(c, rows, cluster, bytes);
            if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
                return BCA_ERR_CUDA;
        }
    return BCA_OK;
}

int launch_paged_rows(const PagedCache &c, const PagedArgs &a, int items, cudaStream_t stream) {
    int bytes = 0;
    const void *f = rows_kernel(c, a.rows, items > 0, bytes);
    PagedArgs args = a;
    void *params[] = {&args};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items > 0 ? items * kCluster : paged_shares(a.rows)));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kCluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = items > 0 ? 1 : 0;
    return cudaLaunchKernelExC(&cfg, f, params) == cudaSuccess ? BCA_OK : BCA_ERR_CUDA;
}

}  // namespace bca
