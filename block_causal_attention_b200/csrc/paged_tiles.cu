// Attention of many packed rows (chunks of new tokens) over the pages of a KV cache.
//
// The mathematics of paged_rows.cu.  Bound by the special-function units: one exponential a
// score, 16 a clock and multiprocessor, against 4 D operations on tensor cores that would do
// twice that many scores.  So the exponentials must never wait:
//   - S = Q K^T by tcgen05.mma (128 x 128 tiles, fp32 in tensor memory), issued by one thread
//     that runs ahead: three tiles of 128 rows share each page, four S tiles go round;
//   - S comes back to the registers in the fragment layout of the warps' matrix instruction
//     (tcgen05.ld.16x256b), so that P needs no way through shared or tensor memory: O += P V
//     is a warp's own mma.sync with O in registers.  A PV product by tcgen05 would have N = D,
//     at most 48, which one thread issues every 45 cycles (N = 128: every 65), and its completion
//     would stand between two softmax steps; here a softmax warp waits for one thing a page, its
//     next S, which has been ready for long;
//   - 12 softmax warps, three a scheduler, with the products of one step between the exponentials
//     of the next, so that both units are at work under every warp;
//   - no running maximum where every row sees the whole page: the sums of the weights, needed
//     anyway, tell when the reference has to move (3.1 -> 2.4 ms at the size below).
// The same instructions without barriers take 1,280 cycles a 128 x 128 tile at D = 24 and 1,480
// at D = 48 (1,024 of them exponentials), this kernel 1,400 and 1,760.  Measured on the
// device: 10,800 tokens of 16 heads over 32,400 keys, D = 48, 2.20 ms, 489 TFLOP/s, the
// special-function units 57 % and the tensor pipe 53 % busy; 6,144 tokens of 32 heads over 13,824
// keys, D = 24, 0.88 ms.  (The dense forward of this library, P V by tcgen05, takes 2.08 and 1.08 ms.)
#include <cuda_runtime.h>

#include <type_traits>

#include "paged_device.cuh"
#include "paged_mma.cuh"

namespace bca {

using namespace sm100;

namespace {

// SL: 128-row tiles that share a page.  Three make a block that fills a multiprocessor; with one,
// for slices of 65 to 256 rows, two blocks share it (a block of three with one tile at work had a
// softmax warp a scheduler: 114 against 83 us for 16 sequences of 8,000 tokens, 128 rows each).
//
// LO: fp16 values and a prologue.  There a query rounded to fp16 after QK-Norm and RoPE would cost
// as much again as the roundings of P and of O (0.00036 against 0.00021 of plain fp32 relative to
// |O|), so what the rounding leaves is kept too, as a second fp16 tile, and S gets both products:
// 0.00029, for 400 us as before (24 heads over 6 ragged sequences, D = 32), 945 against 882 (6,144 new
// tokens over 18,432, D = 24) and 2,455 against 2,199 (10,800 over 32,400, D = 48).  Beside bf16's
// roundings it would not show, and queries given post-prologue are exact; those keep the single tile
// by a template argument, since a branch in the kernel cost them 12 %.
template <int D, int SL, bool LO>
struct TilesSmem {
    static constexpr int ROWS = 128 * SL;
    static constexpr int BUFFERS = SL == 1 ? 2 : 4;  // S tiles of 128 x 128 in tensor memory, used in turn
    static constexpr int THREADS = 128 + 128 * SL;
    static constexpr int DPAD = Geo<D>::DPAD;
    static constexpr int TILE = D * kPage * 2;       // bytes of a page's K or V of one head
    static constexpr int KSTAGE = DPAD * kPage * 2;  // K is padded to whole 16-channel steps
    static constexpr int STAGE = KSTAGE + TILE;
    static constexpr int STAGES = SL == 1 ? (D == 48 ? 3 : 5) - (LO && D >= 32 ? 1 : 0)
                                          : D == 48 ? (LO ? 3 : 6) : D == 32 && LO ? 7 : 8;
    static constexpr int Q_BYTES = 128 * DPAD * 2;
    static constexpr int OFF_Q = 0;
    static constexpr int Q_TILE = (LO ? 2 : 1) * Q_BYTES;  // of 128 rows
    static constexpr int Q_ITEM = SL * Q_TILE;
    static constexpr int OFF_RING = 2 * Q_ITEM;      // queries of this item and of the next
    static constexpr int OFF_BAR = OFF_RING + STAGES * STAGE;
    static constexpr int B_FULL = 0;
    static constexpr int B_EMPTY = STAGES;
    static constexpr int B_ITEM = 2 * STAGES;
    static constexpr int B_S_FULL = B_ITEM + 2 * kItemRing;
    static constexpr int B_S_FREE = B_S_FULL + SL * BUFFERS;  // full: of a slot's use of a buffer
    static constexpr int B_Q_FULL = B_S_FREE + BUFFERS;
    static constexpr int B_Q_FREE = B_Q_FULL + 2;
    static constexpr int B_Q_FIRST = B_Q_FREE + 2;
    static constexpr int B_DONE = B_Q_FIRST + 1;
    static constexpr int OFF_HERE = OFF_BAR + 8 * (B_DONE + 1);
    static constexpr int OFF_TMEM = OFF_HERE + 4 * STAGES;
    static constexpr int OFF_ITEMS = OFF_TMEM + 4;
    static constexpr int OFF_LIMIT = OFF_ITEMS + kItemRing * (int)sizeof(PagedItem);  // of each row
    static constexpr int OFF_ABORT = OFF_LIMIT + 4 * ROWS;
    static constexpr int BYTES = OFF_ABORT + 4;
};

constexpr int kChunk = 32;                 // keys a softmax step takes: 32 scores a thread
constexpr int kTiles = kChunk / 8;

// Lane (g, t) of the warp gets row g, columns 8 n + 2 t and + 1 in f[n][0], f[n][1] and row
// g + 8 in f[n][2], f[n][3]: the accumulator layout of mma.m16n8k16.
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&f)[4][4]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 16; ++i) f[i / 4][i % 4] = __uint_as_float(r[i]);
}

// QK-Norm and RoPE of 16 packed rows of an item, from row `first` on, into the A operand of
// S = Q K^T (fp16, K-major core matrices, tiles of 128 rows); a warp, eight lanes a row.
template <int D, typename T, bool LO>
__device__ __forceinline__ void query_rows(const PagedArgs &a, const PagedItem &x, const float2 (&gain)[Row8<D>::N],
                                           uint8_t *to, int first) {
    using L = TilesSmem<D, 1, LO>;
    const int e = threadIdx.x & 7, r0 = first + (threadIdx.x >> 3 & 3);
    Row8<D> q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t packed = x.head + min(r0 + 4 * i, x.left - 1);
        const int64_t row = x.row + x.token + (int32_t)(packed / a.group);
        q[i].load(static_cast<const T *>(a.q) + (row * a.hq + x.g * a.group + packed % a.group) * D,
                  LO || a.pos ? a.pos + row * 3 : static_cast<const int32_t *>(a.q), e);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + 4 * i;
        if (LO || a.pos) q[i].prologue(gain, a.turns, a.eps, e);
#pragma unroll
        for (int k = 0; k < Row8<D>::N; ++k) {
            const int pr = e + 8 * k;
            if (pr < D / 2) {
                uint8_t *at = to + r / 128 * L::Q_TILE + (pr >> 2) * 2048 + r % 128 * 16 + (pr & 3) * 4;
                const float2 y = r < x.left ? q[i].x[k] : float2{0.f, 0.f};
                const uint32_t hi = pack_f16x2(y.x, y.y);
                *reinterpret_cast<uint32_t *>(at) = hi;
                if constexpr (LO) {
                    const float2 back = Io<__half>::unpack(hi);
                    *reinterpret_cast<uint32_t *>(at + L::Q_BYTES) = pack_f16x2(y.x - back.x, y.y - back.y);
                }
            }
        }
    }
}

template <int D, typename T, int SL, bool LO>
__global__ void __launch_bounds__(128 + 128 * SL, SL == 1 ? 2 : 1)
    paged_tiles_kernel(const __grid_constant__ PagedArgs a) {
    using L = TilesSmem<D, SL, LO>;
    constexpr int kSlots = SL, kBuffers = L::BUFFERS, kRows = L::ROWS, kThreads = L::THREADS;
    constexpr int S = L::STAGES;
    constexpr int NV = D / 8;
    constexpr uint32_t IDESC = idesc_f32acc(128, 128, kFmtF16);
    constexpr float kShift = Io<T>::kShift;

    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t sbase = smem_u32(smem);
    auto bar = [&](int i) -> uint32_t { return sbase + L::OFF_BAR + 8u * (uint32_t)i; };
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::OFF_ABORT);
    volatile int *here = reinterpret_cast<volatile int *>(smem + L::OFF_HERE);
    PagedItem *items = reinterpret_cast<PagedItem *>(smem + L::OFF_ITEMS);
    uint32_t *tmem_ptr = reinterpret_cast<uint32_t *>(smem + L::OFF_TMEM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int c = blockIdx.x;

    if (threadIdx.x == 0) {
        *abort_flag = 0;
        for (int i = 0; i < S; ++i) {
            mbar_init(bar(L::B_FULL + i), 1);
            mbar_init(bar(L::B_EMPTY + i), 4 * kSlots);
        }
        for (int i = 0; i < kSlots * kBuffers; ++i) mbar_init(bar(L::B_S_FULL + i), 1);
        for (int i = 0; i < kBuffers; ++i) mbar_init(bar(L::B_S_FREE + i), 4);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(L::B_Q_FULL + i), 2);
            mbar_init(bar(L::B_Q_FREE + i), 1);
        }
        for (int i = 0; i < kItemRing; ++i) {
            mbar_init(bar(L::B_ITEM + i), 1);
            mbar_init(bar(L::B_ITEM + kItemRing + i), 3 + 4 * kSlots);  // warps 1, 2, 3 and the softmax's
        }
        mbar_init(bar(L::B_Q_FIRST), 4 * kSlots);
        mbar_init(bar(L::B_DONE), 1);
        mbar_fence_init();
    }
    if constexpr (L::DPAD > D) {
        // channels that do not exist: zero in Q and, so that 0 times them is 0, in every K stage
        constexpr int N = (L::KSTAGE - L::TILE) / 16;
        for (int i = threadIdx.x; i < (S + 2 * L::Q_ITEM / L::Q_BYTES) * N; i += kThreads) {
            uint8_t *to = i / N < S ? smem + L::OFF_RING + i / N * L::STAGE + L::TILE
                                    : smem + L::OFF_Q + (i / N - S) * L::Q_BYTES + 128 * D * 2;
            reinterpret_cast<uint4 *>(to)[i % N] = make_uint4(0, 0, 0, 0);
        }
    }
    fence_proxy_async_smem();
    if (warp == 2) {
        tmem_alloc(smem_u32(tmem_ptr), 128 * kBuffers);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = *tmem_ptr;

    // Registers: threads x 128 at launch; the softmax warps take 152 (48 sums of O and 32 scores
    // among them), 128 x 56 + 384 x 152 = 512 x 128, or 200, 128 x 56 + 128 x 200 = 256 x 128.
    if (warp < 4) regs_dec<56>();
    if (warp == 0) {
        paged_fill<kRows, S, L::TILE, L::KSTAGE, L::STAGE>(a, c, sbase + L::OFF_RING, bar(L::B_FULL),
                                                    bar(L::B_ITEM), items, here, abort_flag);
    } else if (warp == 1) {
        // ------------------------------------------------ S = Q K^T
        uint32_t queries = 0;  // items with pages so far
        if (lane == 0) {
            int it = 0;
            uint32_t made = 0;     // S tiles so far
            bool ok = true;
            for (int n = 0; ok; ++n) {
                ok = paged_wait(bar(L::B_ITEM + n % kItemRing), (n / kItemRing) & 1, a, abort_flag);
                if (!ok) break;
                const int32_t p0 = items[n % kItemRing].p0, p1 = items[n % kItemRing].p1;
                const int32_t left = items[n % kItemRing].left;
                if (p0 < 0) break;
                mbar_arrive(bar(L::B_ITEM + kItemRing + n % kItemRing));
                if (p0 == p1) continue;
                const uint32_t qb = queries % 2;
                // (buffer 0 is first filled by the softmax warps, which have a barrier of their own)
                ok = queries == 0 ? paged_wait(bar(L::B_Q_FIRST), 0, a, abort_flag)
                                  : paged_wait(bar(L::B_Q_FULL + qb), (queries / 2 - (qb == 0)) & 1, a, abort_flag);
                ++queries;
                for (int32_t p = p0; p < p1 && ok; ++p, ++it) {
                    const int st = it % S;
                    ok = paged_wait(bar(L::B_FULL + st), (it / S) & 1, a, abort_flag);
#pragma unroll
                    for (int s = 0; s < kSlots; ++s) {
                        if (!ok || s * 128 >= left) continue;
                        const uint32_t buf = made % kBuffers;
                        if (made >= kBuffers)
                            ok = paged_wait(bar(L::B_S_FREE + buf), (made / kBuffers - 1) & 1, a, abort_flag);
                        if (!ok) continue;
                        ++made;
                        tc_fence_after();
                        const uint32_t qa = sbase + L::OFF_Q + qb * L::Q_ITEM + s * L::Q_TILE;
                        const uint32_t kb = sbase + L::OFF_RING + st * L::STAGE;
#pragma unroll
                        for (int k = 0; k < L::DPAD / 16; ++k)
                            mma_f16(tbase + 128 * buf, smem_desc(qa + k * 4096, 2048, 128),
                                    smem_desc(kb + k * 4096, 2048, 128), IDESC, k > 0);
                        if constexpr (LO)
#pragma unroll
                            for (int k = 0; k < L::DPAD / 16; ++k)
                                mma_f16(tbase + 128 * buf, smem_desc(qa + L::Q_BYTES + k * 4096, 2048, 128),
                                        smem_desc(kb + k * 4096, 2048, 128), IDESC, 1);
                        mma_commit(bar(L::B_S_FULL + s * kBuffers + buf));
                    }
                }
                mma_commit(bar(L::B_Q_FREE + qb));
            }
        }
        if (lane == 0) {
            // all issued products must be complete before the tensor memory is given back, and all
            // arrivals made before the barriers' memory is
            mma_commit(bar(L::B_DONE));
            bool done = mbar_wait(bar(L::B_DONE), 0, a.timeout_ns);
            for (uint32_t b = 0; b < 2; ++b) {
                const uint32_t uses = (queries + 1 - b) / 2;
                if (uses > 0) done = done && mbar_wait(bar(L::B_Q_FREE + b), (uses - 1) & 1, a.timeout_ns);
            }
            if (!done) {
                atomicOr(a.status, kPagedTimeout);
                *abort_flag = 1;
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        // ------------------------------------------------ queries, an item ahead
        // Two warps, 32 rows at a time, beside the softmax of the item before.  The block's first
        // item has nothing to hide behind: all softmax warps make its queries.
        const int e = lane & 7;
        float2 gain[Row8<D>::N];
        Row8<D>::load_gain(a.q_gain, e, gain);
        uint32_t queries = 0;
        for (int n = 0;; ++n) {
            if (!__all_sync(0xffffffffu,
                            paged_wait(bar(L::B_ITEM + n % kItemRing), (n / kItemRing) & 1, a, abort_flag)))
                break;
            const PagedItem &x = items[n % kItemRing];
            const int32_t p0 = x.p0, p1 = x.p1;
            if (p0 < 0) break;
            if (p0 < p1) {
                const uint32_t qb = queries % 2;
                if (queries >= 2 && !__all_sync(0xffffffffu, paged_wait(bar(L::B_Q_FREE + qb), (queries / 2 - 1) & 1, a,
                                                                        abort_flag)))
                    break;
                ++queries;
                if (queries > 1) {
                    const int rows = min((x.left + 127) / 128 * 128, kRows);
#pragma unroll 1
                    for (int r = (warp - 2) * 16; r < rows; r += 32)
                        query_rows<D, T, LO>(a, x, gain, smem + L::OFF_Q + qb * L::Q_ITEM, r);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(L::B_Q_FULL + qb));
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(L::B_ITEM + kItemRing + n % kItemRing));
        }
        __syncwarp();
    } else {
        regs_inc<SL == 1 ? 200 : 152>();
        // ------------------------------------------------ softmax and O += P V
        const int slot = (warp - 4) >> 2, quarter = warp & 3;
        const int g = lane >> 2, t = lane & 3;
        const uint32_t tlane = tbase + ((uint32_t)(quarter * 32) << 16);
        // rows 8 j .. of matrix j: V's token group j % 2, channel group j / 2
        const uint32_t vaddr = ((lane >> 3 & 1) * D + 8 * (lane >> 4) + (lane & 7)) * 16;
        int it = 0;
        uint32_t made = 0;                         // S tiles before this item
        // Parity of the next use of each buffer by this slot.  The slots take turns with the
        // buffers, so a barrier of a buffer alone would run through phases that this warp does not
        // wait for, and its parity would tell it nothing.
        uint32_t parity = 0;
        bool first = true;
        bool ok = true;
        const int wr = slot * 128 + quarter * 32;  // the warp's first row of the work tile
        int32_t *limits = reinterpret_cast<int32_t *>(smem + L::OFF_LIMIT) + wr;  // of this warp's rows
        for (int n_item = 0; ok; ++n_item) {
            const uint32_t done = bar(L::B_ITEM + kItemRing + n_item % kItemRing);
            ok = __all_sync(0xffffffffu, paged_wait(bar(L::B_ITEM + n_item % kItemRing), (n_item / kItemRing) & 1, a,
                                                    abort_flag));
            if (!ok) break;
            const PagedItem &x = items[n_item % kItemRing];
            const int32_t p0 = x.p0, p1 = x.p1;
            if (p0 < 0) break;
            if (first && p0 < p1) {
                first = false;
                float2 gain[Row8<D>::N];
                Row8<D>::load_gain(a.q_gain, lane & 7, gain);
#pragma unroll 1
                for (int r = wr; r < wr + 32; r += 16) query_rows<D, T, LO>(a, x, gain, smem + L::OFF_Q, r);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::B_Q_FIRST));
            }
            const int active = (x.left + 127) / 128;  // slots that have rows
            if (slot * 128 >= x.left) {
                for (int32_t p = p0; p < p1 && ok; ++p, ++it) {
                    ok = __all_sync(0xffffffffu, paged_wait(bar(L::B_FULL + it % S), (it / S) & 1, a, abort_flag));
                    if (ok && lane == 0) mbar_arrive(bar(L::B_EMPTY + it % S));
                }
                made += (p1 - p0) * active;
                __syncwarp();
                if (lane == 0) mbar_arrive(done);
                continue;
            }

            float o[2][NV][4], ref[2][2], sum[2][2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
#pragma unroll
                for (int n = 0; n < NV; ++n)
#pragma unroll
                    for (int j = 0; j < 4; ++j) o[m][n][j] = 0.f;
                ref[m][0] = ref[m][1] = -INFINITY;
                sum[m][0] = sum[m][1] = 0.f;
            }
            // keys that all, and that some of the warp's rows see end here
            limits[lane] = x.limit(wr + lane, a.group);
            __syncwarp();
            const int32_t lim_all = x.limit(min(wr, x.left - 1), a.group);
            const int32_t lim_any = x.limit(min(wr + 31, x.left - 1), a.group);
            const int32_t kb = x.kb;
            bool settled = false;  // every row of the warp has a reference
            uint32_t tile = made + slot;   // this warp's S tile: buffer tile % kBuffers
            made += (p1 - p0) * active;
            float s[2][kTiles][4];
            uint32_t pa[2][kTiles / 2][4];  // P of a step as A operands: [16-row tile][16 keys]
            auto load_s = [&](int step) {
                const uint32_t at = tlane + 128 * (tile % kBuffers) + kChunk * step;
                tmem_ld_frag(at, s[0]);
                tmem_ld_frag(at + (16u << 16), s[1]);
            };
            auto wait_s = [&] {
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8 * kTiles; ++i)
                    asm volatile("" : "+f"(s[i / (4 * kTiles)][i / 4 % kTiles][i % 4]));
            };
            auto free_s = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::B_S_FREE + tile % kBuffers));
            };
            auto free_page = [&](int st) {
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(L::B_EMPTY + st));
            };
            // Keys and values of page `it` and the warp's S of them.
            auto wait_page = [&] {
                const uint32_t buf = tile % kBuffers;
                if (ok)
                    ok = __all_sync(0xffffffffu, paged_wait(bar(L::B_FULL + it % S), (it / S) & 1, a, abort_flag) &&
                                                     paged_wait(bar(L::B_S_FULL + slot * kBuffers + buf),
                                                                parity >> buf & 1, a, abort_flag));
                parity ^= 1u << buf;
                tc_fence_after();
                return ok;
            };
            auto page_v = [&](int st) { return sbase + L::OFF_RING + st * L::STAGE + L::KSTAGE; };
            // P = 2^(scale s - ref) of 16 rows x 16 keys, and the sums
            auto weights = [&](int m, int k, uint32_t (&to)[4], float2 (&add)[2]) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float neg = ref[m][h] == -INFINITY ? 0.f : -ref[m][h];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float *x = &s[m][2 * k + b][2 * h];
                        float2 y = fma2(make_float2(x[0], x[1]), make_float2(a.scale, a.scale), make_float2(neg, neg));
                        y = make_float2(ex2(y.x), ex2(y.y));
                        add[h] = b == 0 && k == 0 ? y : add2(add[h], y);
                        to[2 * b + h] = Io<T>::pack(y.x, y.y);
                    }
                }
            };
            // A step in which every row sees every key.  The maxima are not looked at: weights may
            // grow to kTop before the reference has to move, and their sums, which are needed
            // anyway, tell.  The P V products of the step before stand between its exponentials, so
            // that a warp alone keeps both units at work.  False, with s still to be had from tensor
            // memory, if the reference has to move.
            auto fast_step = [&](bool before, uint32_t vs, int vstep) {
                uint32_t pn[2][kTiles / 2][4];
                float2 add[2][2];
#pragma unroll
                for (int k = 0; k < kChunk / 16; ++k) {
                    uint32_t vf[NV][2];
                    if (before) ldsm_v<NV>(vs + (vstep * kTiles + 2 * k) * (D * 16) + vaddr, vf);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        weights(m, k, pn[m][k], add[m]);
                        if (before)
#pragma unroll
                            for (int n = 0; n < NV; ++n) mma16<Io<T>::kF16>(o[m][n], pa[m][k], vf[n][0], vf[n][1]);
                    }
                }
                bool high = false;
                float row[2][2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        row[m][h] = add[m][h].x + add[m][h].y;
                        high |= row[m][h] > Io<T>::kTop;
                    }
                if (__any_sync(0xffffffffu, high)) return false;
#pragma unroll
                for (int m = 0; m < 2; ++m) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) sum[m][h] += row[m][h];
#pragma unroll
                    for (int k = 0; k < kChunk / 16; ++k)
#pragma unroll
                        for (int j = 0; j < 4; ++j) pa[m][k][j] = pn[m][k][j];
                }
                return true;
            };
            auto products = [&](uint32_t vs, int vstep, int k) {  // the 16 keys k of a step
                uint32_t vf[NV][2];
                ldsm_v<NV>(vs + (vstep * kTiles + 2 * k) * (D * 16) + vaddr, vf);
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int n = 0; n < NV; ++n) mma16<Io<T>::kF16>(o[m][n], pa[m][k], vf[n][0], vf[n][1]);
            };
            constexpr int kSteps = kPage / kChunk;

            for (int32_t p = p0; p < p1; ++p, ++it, tile += active) {
                if (!wait_page()) break;
                int32_t page0 = p * kPage;
                bool on = here[it % S];
                int step = 0;
                if (on && settled && page0 >= kb && page0 + kPage <= lim_all) {
                    load_s(0);
                    wait_s();
                    if (fast_step(false, 0, 0)) {
                        // the products of step - 1 are still to be made
                        for (;;) {
                            const uint32_t vs = page_v(it % S);
                            load_s(1);
#pragma unroll
                            for (step = 1; step < kSteps; ++step) {
                                wait_s();
                                if (!fast_step(true, vs, step - 1)) break;
                                if (step + 1 < kSteps) {
                                    load_s(step + 1);
                                } else {
                                    free_s();
                                }
                            }
                            if (step < kSteps) break;
                            // on to the next page, if that one is seen whole too
                            if (p + 1 >= p1 || page0 + 2 * kPage > lim_all) {
                                products(vs, kSteps - 1, 0);
                                products(vs, kSteps - 1, 1);
                                break;
                            }
                            const int old = it % S;
                            ++p, ++it, tile += active;
                            page0 += kPage;
                            if (!wait_page()) break;
                            on = here[it % S];
                            step = 0;
                            if (!on) {
                                products(vs, kSteps - 1, 0);
                                products(vs, kSteps - 1, 1);
                                free_page(old);
                                break;
                            }
                            load_s(0);
                            wait_s();
                            const bool go = fast_step(true, vs, kSteps - 1);
                            free_page(old);
                            if (!go) break;
                        }
                        if (!ok) break;
                    }
                }
                const uint32_t vs = page_v(it % S);
                // Else, or from the step on that passed kTop: step by step, with masks and the running
                // maximum where they are needed.
#pragma unroll 1
                for (; step < kSteps; ++step) {
                    const int32_t key0 = page0 + kChunk * step;
                    const bool work = on && key0 + kChunk > kb && key0 < lim_any;
                    if (work) {
                        load_s(step);
                        wait_s();
                    }
                    const bool inside = key0 >= kb && key0 + kChunk <= lim_all;
                    if (work && inside && settled) {
                        if (fast_step(false, 0, 0)) {
                            if (step == kSteps - 1) free_s();
                            products(vs, step, 0);
                            products(vs, step, 1);
                            continue;
                        }
                        load_s(step);
                        wait_s();
                    }
                    if (step == kSteps - 1) free_s();
                    if (!work) continue;
                    settled = true;
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (!inside) {
                                const int32_t past = limits[16 * m + 8 * h + g] - key0 - 2 * t;
#pragma unroll
                                for (int n = 0; n < kTiles; ++n)
#pragma unroll
                                    for (int j = 0; j < 2; ++j)
                                        if (8 * n + j >= past) s[m][n][2 * h + j] = -INFINITY;
                                if (key0 < kb)
#pragma unroll
                                    for (int n = 0; n < kTiles; ++n)
#pragma unroll
                                        for (int j = 0; j < 2; ++j)
                                            if (8 * n + j < kb - key0 - 2 * t) s[m][n][2 * h + j] = -INFINITY;
                            }
                            float top = s[m][0][2 * h];
#pragma unroll
                            for (int n = 0; n < kTiles; ++n) top = fmaxf(top, fmaxf(s[m][n][2 * h], s[m][n][2 * h + 1]));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)) * a.scale - kShift;
                            if (top > ref[m][h]) {
                                const float mul = ref[m][h] == -INFINITY ? 0.f : ex2(ref[m][h] - top);
                                ref[m][h] = top;
                                sum[m][h] *= mul;
#pragma unroll
                                for (int n = 0; n < NV; ++n) {
                                    o[m][n][2 * h] *= mul;
                                    o[m][n][2 * h + 1] *= mul;
                                }
                            }
                            settled &= ref[m][h] != -INFINITY;
                        }
                    settled = __all_sync(0xffffffffu, settled);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        float2 add[2];
#pragma unroll
                        for (int k = 0; k < kChunk / 16; ++k) weights(m, k, pa[m][k], add);
#pragma unroll
                        for (int h = 0; h < 2; ++h) sum[m][h] += add[h].x + add[h].y;
                    }
#pragma unroll
                    for (int k = 0; k < kChunk / 16; ++k) {
                        const uint32_t at = (step * kTiles + 2 * k) * (D * 16);
                        const int32_t keyk = key0 + 16 * k;
                        uint32_t vf[NV][2];
                        ldsm_v<NV>(vs + at + vaddr, vf);
                        bool odd = false;
                        if (!inside) odd = clear_unseen<T, NV>(vf, keyk + 2 * t, kb, lim_any);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
#pragma unroll
                            for (int n = 0; n < NV; ++n) mma16<Io<T>::kF16>(o[m][n], pa[m][k], vf[n][0], vf[n][1]);
                            if (odd) {
                                int32_t lim[2];
#pragma unroll
                                for (int h = 0; h < 2; ++h) lim[h] = limits[16 * m + 8 * h + g];
                                add_left_out<D, T, NV>(o[m], pa[m][k],
                                                       reinterpret_cast<const T *>(smem + (vs + at - sbase)), keyk, kb,
                                                       lim);
                            }
                        }
                    }
                }
                free_page(it % S);
            }

            // ------------------------------------------------ O / l and the LSE, or this block's piece
            float *part = paged_part(a, D, x.part);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float l = sum[m][h];
                    l += __shfl_xor_sync(0xffffffffu, l, 1);
                    l += __shfl_xor_sync(0xffffffffu, l, 2);
                    const int r = wr + 16 * m + 8 * h + g;
                    if (r >= x.left) continue;
                    if (x.whole) {
                        const bool none = ref[m][h] == -INFINITY && l == 0.f;  // (NaN scores leave a NaN in l)
                        const float inv = none ? 0.f : 1.f / l;
                        const uint32_t packed = x.head + r;
                        const int64_t token = x.row + x.token + (int32_t)(packed / a.group);
                        const int head = x.g * a.group + (int)(packed % a.group);
                        const int64_t at = (token * a.hq + head) * D + 2 * t;
#pragma unroll
                        for (int n = 0; n < NV; ++n) {
                            const float y0 = none ? 0.f : o[m][n][2 * h] * inv;
                            const float y1 = none ? 0.f : o[m][n][2 * h + 1] * inv;
                            if (a.o_fp32)
                                *reinterpret_cast<float2 *>(static_cast<float *>(a.o) + at + 8 * n) = make_float2(y0, y1);
                            else
                                *reinterpret_cast<uint32_t *>(static_cast<T *>(a.o) + at + 8 * n) = Io<T>::pack(y0, y1);
                        }
                        if (a.lse && t == 0)
                            a.lse[head * a.nq + token] = none ? -INFINITY : (ref[m][h] + log2f(l)) * 0.69314718055994531f;
                    } else {  // without pages too: the sum, 0, tells
#pragma unroll
                        for (int n = 0; n < NV; ++n)
                            *reinterpret_cast<float2 *>(part + (size_t)r * D + 8 * n + 2 * t) =
                                make_float2(o[m][n][2 * h], o[m][n][2 * h + 1]);
                        if (t == 0) {
                            part[(size_t)kRows * D + r] = ref[m][h];
                            part[(size_t)kRows * (D + 1) + r] = l;
                        }
                    }
                }
            __syncwarp();
            if (lane == 0) mbar_arrive(done);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tbase, 128 * kBuffers);
    }
}

template <int D, typename T, int SL, bool LO>
const void *tiles_kernel(int &bytes) {
    bytes = TilesSmem<D, SL, LO>::BYTES;
    return (const void *)paged_tiles_kernel<D, T, SL, LO>;
}

template <int D, int SL>
const void *tiles_kernel(bool f16, bool prologue, int &bytes) {
    if (!f16) return tiles_kernel<D, __nv_bfloat16, SL, false>(bytes);
    return prologue ? tiles_kernel<D, __half, SL, true>(bytes) : tiles_kernel<D, __half, SL, false>(bytes);
}

const void *tiles_kernel(const PagedCache &c, int rows, bool prologue, int &bytes) {
    const bool f16 = (c.flags & BCA_PAGED_FP16) != 0, narrow = rows == kPagedNarrowRows;
    switch (c.d) {
        case 24: return narrow ? tiles_kernel<24, 1>(f16, prologue, bytes) : tiles_kernel<24, 3>(f16, prologue, bytes);
        case 32: return narrow ? tiles_kernel<32, 1>(f16, prologue, bytes) : tiles_kernel<32, 3>(f16, prologue, bytes);
        default: return narrow ? tiles_kernel<48, 1>(f16, prologue, bytes) : tiles_kernel<48, 3>(f16, prologue, bytes);
    }
}

}  // namespace

int prepare_paged_tiles(const PagedCache &c) {
    for (int rows : {kPagedNarrowRows, kPagedTileRows})
        for (bool prologue : {false, true}) {
            int bytes = 0;
            const void *f = tiles_kernel(c, rows, prologue, bytes);
            if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
                return BCA_ERR_CUDA;
        }
    return BCA_OK;
}

int launch_paged_tiles(const PagedCache &c, const PagedArgs &a, cudaStream_t stream) {
    int bytes = 0;
    const void *f = tiles_kernel(c, a.rows, a.pos != nullptr, bytes);
    PagedArgs args = a;
    void *params[] = {&args};
    return cudaLaunchKernel(f, dim3((unsigned)paged_shares(a.rows)), dim3((unsigned)(128 + a.rows)), params,
                            (size_t)bytes, stream) == cudaSuccess
               ? BCA_OK
               : BCA_ERR_CUDA;
}

}  // namespace bca
