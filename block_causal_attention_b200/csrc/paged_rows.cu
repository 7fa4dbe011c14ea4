// Attention of few packed rows (single tokens, proposed tokens, small groups) over the pages
// of a KV cache.
//
// O_i = sum_j 2^(s_ij - r_i) v_j / sum_j 2^(s_ij - r_i), s_ij = log2(e)/sqrt(D) q_i . k_j, in
// one pass over the keys: the reference r_i follows the running maximum.
//
// Bound by memory: a key and value of a KV head are 4 D bytes for 4 D * rows operations, so at
// 16 to 64 rows even the warps' own matrix instructions keep up.  What counts is bytes in
// flight: one block a multiprocessor, a ring of whole pages (a page's keys and values of one
// head are two contiguous stretches, moved by two bulk copies) filled by one warp that runs
// ahead over page and item borders.  Eight warps take 16 of a page's 128 tokens each; their
// results meet once an item, so that one page is enough work for all of them.
//
// The layout of the pages is that of the 8 x 8 matrices that ldmatrix reads: 8 tokens x 8
// channels of K and 8 channels x 8 tokens of V lie in 128 contiguous bytes, so both operands
// come to the registers without bank conflicts and without a transposition.
#include <cuda_runtime.h>

#include <type_traits>

#include "paged_device.cuh"

namespace bca {

using namespace sm100;

namespace {

constexpr int kWarps = 8;                     // consumers; one more fills the ring
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kWarpTokens = kPage / kWarps;   // 16

template <int D>
struct RowsSmem {
    static constexpr int TILE = D * kPage * 2;
    static constexpr int STAGES = D == 48 ? 7 : D == 32 ? 10 : 13;
    static constexpr int QSTRIDE = D == 24 ? 40 : D + 8;  // elements; an odd number of 16-byte units
    static constexpr int OFF_RING = 0;
    static constexpr int OFF_Q = STAGES * 2 * TILE;
    static constexpr int OFF_MERGE = OFF_Q + 64 * QSTRIDE * 2;
    static constexpr int OFF_BAR = OFF_MERGE + kWarps * 16 * (D + 2) * 4;
    static constexpr int OFF_HERE = OFF_BAR + 2 * STAGES * 8;
    static constexpr int OFF_ABORT = OFF_HERE + STAGES * 4;
    static constexpr int BYTES = OFF_ABORT + 4;
};

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm2(uint32_t addr, uint32_t &r0, uint32_t &r1) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}

// c += a b, 16 x 8 x 16, fp32 sums
template <bool F16>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma8_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b0) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5}, {%6}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(b0));
}

// MT: 16-row matrix tiles a work tile has (rows = 16 MT).
template <int D, typename T, int MT>
__global__ void __launch_bounds__(kThreads, 1) paged_rows_kernel(const __grid_constant__ PagedArgs a) {
    using L = RowsSmem<D>;
    constexpr int S = L::STAGES;
    constexpr int R = 16 * MT;
    constexpr int KS = D / 16;            // 16-channel steps; D = 24 has an 8-channel one behind
    constexpr bool TAIL = D % 16 != 0;
    constexpr int NV = D / 8;
    constexpr float kShift = Io<T>::kShift;

    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ PagedLocate sh;
    const uint32_t sbase = smem_u32(smem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    volatile int *here = reinterpret_cast<volatile int *>(smem + L::OFF_HERE);
    auto full = [&](int i) -> uint32_t { return sbase + L::OFF_BAR + 8u * (uint32_t)i; };
    auto empty = [&](int i) -> uint32_t { return sbase + L::OFF_BAR + 8u * (uint32_t)(S + i); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    // the joining kernel may be put in place as blocks of this one end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < S; ++i) {
            mbar_init(full(i), 1);
            mbar_init(empty(i), kWarps);
        }
        mbar_fence_init();
    }
    PagedCursor cur;
    uint64_t lo, hi, total;
    const int c = blockIdx.x;
    if (!paged_locate(a, c, false, sh, lo, hi, total, cur)) return;
    __syncthreads();

    if (warp == kWarps) {
        // ------------------------------------------------ fills the ring
        int it = 0;
        bool ok = !a.skip_loads;
        do {
            int32_t p0, p1;
            cur.pages(a, lo, hi, p0, p1);
            const int32_t *row = a.table + (int64_t)cur.s.b * a.width;
            for (int32_t base = p0; base < p1 && ok; base += 32) {
                const int32_t mine = base + lane < p1 ? __ldg(row + base + lane) : -1;
                const int count = min(32, p1 - base);
                for (int j = 0; j < count; ++j) {
                    const int32_t page = __shfl_sync(0xffffffffu, mine, j);
                    if (lane == 0 && ok) {
                        const int st = it % S;
                        if (it >= S) ok = paged_wait(empty(st), (it / S - 1) & 1, a, abort_flag);
                        if (ok) {
                            const bool on = page >= 0 && page < a.pages;
                            here[st] = on;
                            if (on) {
                                const int64_t at = ((int64_t)page * a.hkv + cur.g) * L::TILE;
                                const uint32_t dst = sbase + L::OFF_RING + st * 2 * L::TILE;
                                mbar_arrive_expect_tx(full(st), 2 * L::TILE);
                                bulk_g2s(dst, static_cast<const uint8_t *>(a.k_pages) + at, L::TILE, full(st));
                                bulk_g2s(dst + L::TILE, static_cast<const uint8_t *>(a.v_pages) + at, L::TILE,
                                         full(st));
                            } else {
                                mbar_arrive(full(st));
                            }
                            ++it;
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
            }
        } while (ok && cur.end() < hi && cur.next(a));
        // every copy must have landed before the block may end
        if (lane == 0)
            for (int j = it > S ? it - S : 0; j < it; ++j)
                if (!mbar_wait(full(j % S), (j / S) & 1, a.timeout_ns)) {
                    atomicOr(a.status, kPagedTimeout);
                    *abort_flag = 1;
                }
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
    bool ok = true;
    int it = 0;
    do {
        int32_t p0, p1;
        cur.pages(a, lo, hi, p0, p1);
        const bool whole = lo <= cur.start && cur.end() <= hi;

        // queries: QK-Norm and RoPE, fp16 (|q_hat| <= sqrt(D) max|gain|; 11 bits of significand
        // against bf16's 8).  The softmax scale is applied to the scores in fp32 instead, so that
        // bf16 queries given post-prologue stay exact.
        for (int r = threadIdx.x >> 3; r < R; r += kWarps * 4) {
            const int64_t packed = cur.t * R + r;
            const int64_t token = packed / a.group;
            const int e = lane & 7;
            Row8<D> x;
            const bool live = token < cur.s.n;  // the same for the eight lanes of a row
            const int64_t row = cur.s.r0 + (live ? token : 0);
            x.load(static_cast<const T *>(a.q) + (row * a.hq + cur.g * a.group + packed % a.group) * D, e);
            if (a.pos) x.prologue(a.pos + row * 3, a.q_gain, a.turns, a.eps, e);
#pragma unroll
            for (int i = 0; i < Row8<D>::N; ++i)
                if (e + 8 * i < D / 2)
                    *reinterpret_cast<uint32_t *>(qs + r * L::QSTRIDE + 2 * (e + 8 * i)) =
                        live ? pack_f16x2(x.x[i].x, x.x[i].y) : 0u;
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
            for (int h = 0; h < 2; ++h) {
                const int64_t token = (cur.t * R + 16 * m + g + 8 * h) / a.group;
                lim[m][h] = token < cur.s.n ? paged_limit(a, cur.s, (int32_t)token) : 0;
            }
        }
        // keys that every row of the tile sees end here, and those that any row sees there
        const int32_t lim_all = paged_limit(a, cur.s, (int32_t)(cur.t * R / a.group));
        const int32_t lim_any = paged_limit(
            a, cur.s, (int32_t)min(((cur.t + 1) * R - 1) / a.group, (int64_t)cur.s.n - 1));

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
            if (here[st] && key0 + kWarpTokens > cur.s.kb && key0 < lim_any) {
                const uint32_t ks = sbase + L::OFF_RING + st * 2 * L::TILE, vs = ks + L::TILE;
                uint32_t kf[KS][4], kt[2] = {0, 0}, vf[NV][2];
#pragma unroll
                for (int k = 0; k < KS; ++k) ldsm4(ks + kaddr + k * (2 * kPage * 16), kf[k]);
                if constexpr (TAIL)
                    ldsm2(ks + KS * (2 * kPage * 16) + (2 * warp + (lane >> 3 & 1)) * 128 + (lane & 7) * 16, kt[0], kt[1]);
#pragma unroll
                for (int n = 0; n + 1 < NV; n += 2) {
                    uint32_t r[4];
                    ldsm4(vs + vaddr + n * 128, r);
                    vf[n][0] = r[0];
                    vf[n][1] = r[1];
                    vf[n + 1][0] = r[2];
                    vf[n + 1][1] = r[3];
                }
                if constexpr (NV % 2 == 1) ldsm2(vs + vaddr + (NV - 1) * 128, vf[NV - 1][0], vf[NV - 1][1]);

                const bool inside = key0 >= cur.s.kb && key0 + kWarpTokens <= lim_all;
                bool odd = false;  // values that are not finite, at keys that some rows do not see
                if (!inside) {
                    // a weight of 0 does not silence a NaN or an infinity: what no row sees is cleared
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const int32_t key = key0 + 8 * b + 2 * t;
                        const uint32_t keep = (key >= cur.s.kb && key < lim_any ? 0xffffu : 0u) |
                                              (key + 1 >= cur.s.kb && key + 1 < lim_any ? 0xffff0000u : 0u);
#pragma unroll
                        for (int n = 0; n < NV; ++n) {
                            uint32_t v = vf[n][b] & keep;
                            if (Io<T>::bad(v)) {
                                odd = true;
                                v &= 0xffff0000u;
                            }
                            if (Io<T>::bad(v >> 16)) {
                                odd = true;
                                v &= 0xffffu;
                            }
                            vf[n][b] = v;
                        }
                    }
                    odd = __any_sync(0xffffffffu, odd);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    float s[2][4] = {};
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        mma16<true>(s[0], qa[m][k], kf[k][0], kf[k][1]);
                        mma16<true>(s[1], qa[m][k], kf[k][2], kf[k][3]);
                    }
                    if constexpr (TAIL) {
                        mma8_f16(s[0], qt[m][0], qt[m][1], kt[0]);
                        mma8_f16(s[1], qt[m][0], qt[m][1], kt[1]);
                    }
                    if (!inside) {
#pragma unroll
                        for (int n = 0; n < 2; ++n)
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const int32_t key = key0 + 8 * n + 2 * t + (j & 1);
                                if (key < cur.s.kb || key >= lim[m][j >> 1]) s[n][j] = -INFINITY;
                            }
                    }
                    float mx[2];
                    mx[0] = fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1])) * a.scale;
                    mx[1] = fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3])) * a.scale;
                    const bool grow = mx[0] > ref[m][0] + (kShift + kLazy) || mx[1] > ref[m][1] + (kShift + kLazy);
                    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            float top = mx[h];
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
                    const float sub[2] = {ref[m][0] == -INFINITY ? 0.f : ref[m][0],
                                          ref[m][1] == -INFINITY ? 0.f : ref[m][1]};
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            s[n][j] = ex2(fmaf(s[n][j], a.scale, -sub[j >> 1]));
                            sum[m][j >> 1] += s[n][j];
                        }
                    // P in the values' type: it is a factor of the matrix product
                    const uint32_t pa[4] = {Io<T>::pack(s[0][0], s[0][1]), Io<T>::pack(s[0][2], s[0][3]),
                                            Io<T>::pack(s[1][0], s[1][1]), Io<T>::pack(s[1][2], s[1][3])};
#pragma unroll
                    for (int n = 0; n < NV; ++n) mma16<Io<T>::kF16>(o[m][n], pa, vf[n][0], vf[n][1]);
                    if (odd) {
                        // the values left out above, for the rows that do see their key
                        const T *v = reinterpret_cast<const T *>(smem + L::OFF_RING + st * 2 * L::TILE + L::TILE);
#pragma unroll 1
                        for (int x = 0; x < kWarpTokens; ++x) {
                            const int src = (lane & ~3) + (x % 8) / 2;
                            float w[2];
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float even = __shfl_sync(0xffffffffu, x < 8 ? s[0][2 * h] : s[1][2 * h], src);
                                const float odd_ = __shfl_sync(0xffffffffu, x < 8 ? s[0][2 * h + 1] : s[1][2 * h + 1], src);
                                w[h] = x % 2 ? odd_ : even;
                            }
                            const int32_t key = key0 + x;
#pragma unroll
                            for (int n = 0; n < NV; ++n)
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    const T y = v[((2 * warp + x / 8) * D + 8 * n + 2 * t + (j & 1)) * 8 + x % 8];
                                    if (Io<T>::bad(*reinterpret_cast<const uint16_t *>(&y)) && key >= cur.s.kb &&
                                        key < lim[m][j >> 1])
                                        o[m][n][j] += w[j >> 1] * (float)y;
                                }
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(st));
        }

        // ------------------------------------------------ the eight warps' results meet
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float *mine = merge + warp * 16 * (D + 2);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float l = sum[m][h];
                l += __shfl_xor_sync(0xffffffffu, l, 1);
                l += __shfl_xor_sync(0xffffffffu, l, 2);
                float *row = mine + (g + 8 * h) * (D + 2);
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
                const float *x = row + w * 16 * (D + 2);
                const float mul = top == -INFINITY ? 0.f : ex2(x[D] - top);
                l = fmaf(x[D + 1], mul, l);
#pragma unroll
                for (int i = 0; i < (D + 15) / 16; ++i)
                    if (e + 16 * i < D) y[i] = fmaf(x[e + 16 * i], mul, y[i]);
            }
            const int64_t packed = cur.t * R + 16 * m + r;
            const int64_t token = packed / a.group;
            if (token < cur.s.n) {
                if (whole) {
                    const bool none = top == -INFINITY;
                    const float inv = none ? 0.f : 1.f / l;
                    const int head = cur.g * a.group + (int)(packed % a.group);
                    const int64_t at = ((cur.s.r0 + token) * a.hq + head) * D;
#pragma unroll
                    for (int i = 0; i < (D + 15) / 16; ++i) {
                        if (e + 16 * i >= D) continue;
                        const float z = none ? 0.f : y[i] * inv;
                        if (a.o_fp32) static_cast<float *>(a.o)[at + e + 16 * i] = z;
                        else static_cast<T *>(a.o)[at + e + 16 * i] = T(z);
                    }
                    if (a.lse && e == 0)
                        a.lse[head * a.nq + cur.s.r0 + token] =
                            none ? -INFINITY : (top + log2f(l)) * 0.69314718055994531f;
                } else if (p0 < p1) {
                    float *part = paged_part(a, D, 2 * c + (lo <= cur.start ? 1 : 0));
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
    } while (cur.end() < hi && cur.next(a));
}

template <int D, typename T>
const void *rows_kernel(int rows) {
    switch (rows) {
        case 16: return (const void *)paged_rows_kernel<D, T, 1>;
        case 32: return (const void *)paged_rows_kernel<D, T, 2>;
        default: return (const void *)paged_rows_kernel<D, T, 4>;
    }
}

const void *rows_kernel(const PagedCache &c, int rows, int &bytes) {
    const bool f16 = (c.flags & BCA_PAGED_FP16) != 0;
    switch (c.d) {
        case 24:
            bytes = RowsSmem<24>::BYTES;
            return f16 ? rows_kernel<24, __half>(rows) : rows_kernel<24, __nv_bfloat16>(rows);
        case 32:
            bytes = RowsSmem<32>::BYTES;
            return f16 ? rows_kernel<32, __half>(rows) : rows_kernel<32, __nv_bfloat16>(rows);
        default:
            bytes = RowsSmem<48>::BYTES;
            return f16 ? rows_kernel<48, __half>(rows) : rows_kernel<48, __nv_bfloat16>(rows);
    }
}

}  // namespace

int prepare_paged_rows(const PagedCache &c) {
    for (int rows : {16, 32, 64}) {
        int bytes = 0;
        const void *f = rows_kernel(c, rows, bytes);
        if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
            return BCA_ERR_CUDA;
    }
    return BCA_OK;
}

int launch_paged_rows(const PagedCache &c, const PagedArgs &a, cudaStream_t stream) {
    int bytes = 0;
    const void *f = rows_kernel(c, a.rows, bytes);
    PagedArgs args = a;
    void *params[] = {&args};
    return cudaLaunchKernel(f, dim3((unsigned)a.shares), dim3(kThreads), params, (size_t)bytes, stream) == cudaSuccess
               ? BCA_OK
               : BCA_ERR_CUDA;
}

}  // namespace bca
