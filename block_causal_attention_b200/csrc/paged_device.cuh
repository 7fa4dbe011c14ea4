// Device code shared by the paged-cache kernels: a call's arguments, how its work is cut
// into equal shares, and the QK-Norm + 3D RoPE of rows at explicit positions.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "paged.hpp"
#include "prologue.cuh"
#include "sm100.cuh"

namespace bca {

struct PagedArgs {
    const void *q;
    const int32_t *pos;   // [nq][3], or null: q given post-prologue
    const float *q_gain;
    const void *k_pages, *v_pages;
    const int32_t *table;
    const int32_t *off, *seq, *k_begin, *k_end;  // seq null: slice i reads row i
    void *o;
    float *lse;
    // Pieces of items that several blocks share: slot 2c (block c goes on with an item) and 2c + 1
    // (it begins one that it does not end); a slot is [rows][D] O, [rows] reference, [rows] sum,
    // fp32.  joins[c]: the item of slot 2c + 1.
    float *part;
    struct PagedJoin *joins;
    int *status;
    int64_t nq, pages;
    int seqs, width, slices, causal;
    int hq, hkv, group;
    int rows;             // packed rows of a tile
    int shift;            // a unit of weight is 16 << shift keys
    int o_fp32;
    float eps;
    float scale;          // log2(e) / sqrt(D)
    uint64_t timeout_ns;
    int skip_loads;       // failure-detection test: issue no page loads
    uint64_t turns[24];
};

// ------------------------------------------------------------------ the work and its shares
//
// A slice's queries are packed token by token, the `group` query heads of a KV head next to
// one another, and cut into tiles of `rows` packed rows: the rows of a tile read the same
// keys.  An item is a tile of one KV head.  Items stand in a row (slice, KV head, tile), each
// as long as its weight, about the keys it reads; block c takes the c-th of as many
// equal stretches as there are blocks of that row.  A stretch that ends inside an item splits the item's pages in
// proportion; the pieces are joined by paged_join_kernel.  So the load is even whatever the
// lengths are (they are device data), and the cut depends on the arguments alone: the same
// call gives the same bits.

// Weight of an item that reads no page, in units of 16 << shift keys: its prologue, its epilogue
// and its first page, as measured: one page of the register tiles, two pages of the 384-row
// tiles, four with the causal rule, whose last pages are masked (fitted to the blocks' clocks:
// 8,500 and 17,200 cycles an item beside 4,200 a page; a page of the 128-row tiles takes less).  The whole row of items is below 2^31
// units long (the host picks the shift for the sizes of the call), so all of this is 32-bit
// arithmetic: before a block knows what to load it can do nothing else, and 64-bit divisions
// here took 2 us.
template <int R>
__device__ __forceinline__ uint32_t paged_item_weight(bool causal) {
    return R < kPagedNarrowRows ? 8u : R == kPagedNarrowRows ? (causal ? 40u : 24u) : causal ? 32u : 16u;
}

struct PagedSlice {
    int32_t r0, n;        // its rows of q
    int32_t b;            // table row
    int32_t kb, ke;       // keys [kb, ke) that it sees; kb == ke: none
    int32_t end;          // k_end as given (>= 0): the causal rule counts back from it
    uint32_t tiles;       // of one KV head
    uint32_t w0, dw;      // weight of tile t: w0 + dw * (t + 1), and of the last one
    uint32_t cut;         // this less: a 384-row tile with 128 or 256 rows takes less time

    __device__ __forceinline__ uint32_t upto(uint32_t t) const {  // weight of its first t tiles
        return t * w0 + (dw == 0 ? 0u : dw * (t * (t + 1) / 2)) - (t == tiles ? cut : 0u);
    }
    __device__ __forceinline__ uint32_t weight(uint32_t t) const {
        return w0 + dw * (t + 1) - (t + 1 == tiles ? cut : 0u);
    }
};

template <int R>
__device__ __forceinline__ PagedSlice paged_slice(const PagedArgs &a, int i) {
    PagedSlice s;
    const int32_t nq = (int32_t)a.nq;
    const int32_t o0 = __ldg(a.off + i), o1 = __ldg(a.off + i + 1);
    const int32_t row = __ldg((a.seq ? a.seq : a.off) + i), kb = __ldg(a.k_begin + i), ke = __ldg(a.k_end + i);
    const int32_t b = a.seq ? row : i;
    s.r0 = min(max(o0, 0), nq);
    s.n = min(max(o1, s.r0), nq) - s.r0;
    s.b = b;
    s.end = max(ke, 0);
    s.kb = max(kb, 0);
    s.ke = min(s.end, a.width * kPage);
    if (b < 0 || b >= a.seqs || s.ke <= s.kb) s.kb = s.ke = 0;
    // n * group rows: below 2^32, since Q itself fits a GPU
    s.tiles = ((uint32_t)s.n * (uint32_t)a.group + (R - 1)) / R;
    const int32_t keys = s.ke - s.kb;
    const int unit = 4 + a.shift;
    const uint32_t item = paged_item_weight<R>(a.causal);
    if (a.causal) {
        s.dw = (uint32_t)R / (uint32_t)a.group >> unit;
        s.w0 = item + ((uint32_t)max(keys - s.n, 0) >> unit);
    } else {
        s.dw = 0;
        s.w0 = item + ((uint32_t)keys >> unit);
    }
    s.cut = 0;
    if (R == kPagedTileRows && s.tiles > 0) {
        // a page with one, two, three tiles of 128 rows: 0.55, 0.77, 1 of the time
        const uint32_t slots = ((uint32_t)s.n * (uint32_t)a.group - (s.tiles - 1) * R + 127) / 128;
        s.cut = (s.w0 + s.dw * s.tiles - item) * (3 - slots) / 4;
    }
    return s;
}

// First key that row `token` (counted in the slice) does not see.
__device__ __forceinline__ int32_t paged_limit(const PagedArgs &a, const PagedSlice &s, int32_t token) {
    if (!a.causal) return s.ke;
    return min(s.ke, s.end - (s.n - 1 - token));  // no overflow: both are >= 0 and below 2^31
}

// Where share c begins in a row of this total weight: total * c / shares.
template <int R>
__device__ __forceinline__ uint32_t paged_share(uint32_t total, int c) {
    constexpr uint32_t n = paged_shares(R);
    const uint32_t x = (uint32_t)c;
    return total / n * x + total % n * x / n;
}

template <int R>
struct PagedCursor {
    PagedSlice s;
    int32_t slice;
    int32_t g;          // KV head
    uint32_t t;         // tile
    uint32_t start;     // where the item begins

    __device__ __forceinline__ uint32_t end() const { return start + s.weight(t); }

    // Pages of the item, and the part of them that lies in [lo, hi).  A cut inside the item takes
    // its share of the pages in fp32: any rounding does, as long as it never falls along the item
    // and is the same in the two blocks that meet there.
    __device__ __forceinline__ void pages(const PagedArgs &a, uint32_t lo, uint32_t hi, int32_t &p0,
                                          int32_t &p1) const {
        const uint32_t last = min(((t + 1) * R - 1) / (uint32_t)a.group, (uint32_t)(s.n - 1));
        const int32_t ke = a.causal ? paged_limit(a, s, (int32_t)last) : s.ke;
        const int32_t first = s.kb / kPage;
        const int32_t np = ke > s.kb ? (ke - 1) / kPage + 1 - first : 0;
        const uint32_t w = s.weight(t);
        const float ratio = __fdiv_rn((float)np, (float)w);
        p0 = first + (lo > start ? min(np, (int32_t)__fmul_rn((float)(lo - start), ratio)) : 0);
        p1 = first + (hi < start + w ? min(np, (int32_t)__fmul_rn((float)(hi - start), ratio)) : np);
        p1 = max(p0, p1);
    }

    // The next item (all 32 lanes of a warp together: slices without rows are passed over 32
    // at a time).  False behind the last one.
    __device__ __forceinline__ bool next(const PagedArgs &a) {
        start = end();
        if (++t < s.tiles) return true;
        t = 0;
        if (++g < a.hkv) return true;
        g = 0;
        for (int base = slice + 1; base < a.slices; base += 32) {
            const int i = base + (int)(threadIdx.x & 31);
            bool some = false;
            if (i < a.slices) {
                const int32_t nq = (int32_t)a.nq;
                const int32_t r0 = min(max(__ldg(a.off + i), 0), nq);
                some = min(max(__ldg(a.off + i + 1), r0), nq) > r0;
            }
            const uint32_t m = __ballot_sync(0xffffffffu, some);
            if (m) {
                slice = base + __ffs(m) - 1;
                s = paged_slice<R>(a, slice);
                return true;
            }
        }
        return false;
    }
};

// The stretch [lo, hi) of share c and the item that it begins in, found by one warp, a slice a
// lane at a time.  False when the stretch is empty.
template <int R>
__device__ __forceinline__ bool paged_locate(const PagedArgs &a, int c, uint32_t &lo, uint32_t &hi, uint32_t &total,
                                             PagedCursor<R> &cur) {
    const int lane = threadIdx.x & 31;
    // Up to 32 slices stay in the lanes' registers; of more, four loads are on the way at a time
    // here, and the next 32 while 32 are looked through below.
    PagedSlice s, ahead;
    uint32_t mine = 0, sum = 0;
#pragma unroll 4
    for (int i = lane; i < a.slices; i += 32) {
        s = paged_slice<R>(a, i);
        mine = (uint32_t)a.hkv * s.upto(s.tiles);
        sum += mine;
    }
    total = __reduce_add_sync(0xffffffffu, sum);
    lo = paged_share<R>(total, c);
    hi = paged_share<R>(total, c + 1);
    if (lo == hi) return false;

    // (offsets that do not rise may make the whole longer than 2^32, and then nothing be found)
    uint32_t carry = 0, pre = 0;
    int src = -1;
    if (a.slices > 32) ahead = paged_slice<R>(a, lane);
#pragma unroll 1
    for (int base = 0; base < a.slices && src < 0; base += 32) {
        if (a.slices > 32) {
            s = ahead;
            mine = base + lane < a.slices ? (uint32_t)a.hkv * s.upto(s.tiles) : 0u;
            if (base + 32 + lane < a.slices) ahead = paged_slice<R>(a, base + 32 + lane);
        }
        uint32_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        pre = carry + inc - mine;
        src = __ffs(__ballot_sync(0xffffffffu, pre <= lo && lo - pre < mine)) - 1;
        carry += __shfl_sync(0xffffffffu, inc, 31);
        cur.slice = base + src;
    }
    if (src < 0) return false;
    auto give = [&](auto x) { return __shfl_sync(0xffffffffu, x, src); };
    cur.s.r0 = give(s.r0);
    cur.s.n = give(s.n);
    cur.s.b = give(s.b);
    cur.s.kb = give(s.kb);
    cur.s.ke = give(s.ke);
    cur.s.end = give(s.end);
    cur.s.tiles = give(s.tiles);
    cur.s.w0 = give(s.w0);
    cur.s.dw = give(s.dw);
    cur.s.cut = give(s.cut);
    const uint32_t per_head = cur.s.upto(cur.s.tiles);
    uint32_t rest = lo - give(pre);
    cur.g = (int32_t)(rest / per_head);
    rest -= (uint32_t)cur.g * per_head;
    uint32_t t = 0;
    if (cur.s.tiles > 1) {
        t = rest / cur.s.w0;
        if (cur.s.dw != 0) {
            // upto(t) <= rest, a quadratic in t; the loops take the rounding out
            const float h = (float)cur.s.w0 + 0.5f * cur.s.dw;
            t = (uint32_t)((sqrtf(h * h + 2.0f * cur.s.dw * (float)rest) - h) / cur.s.dw);
        }
        t = min(t, cur.s.tiles - 1);
        while (t > 0 && cur.s.upto(t) > rest) --t;
        while (t + 1 < cur.s.tiles && cur.s.upto(t + 1) <= rest) ++t;
    }
    cur.t = t;
    cur.start = lo - (rest - cur.s.upto(t));
    return true;
}

// Calls of few items over short rows: a cluster of kCluster blocks has an item, the pages in equal
// parts, and joins the parts over distributed shared memory: no shares, no second launch.  Slice i
// has the item slots from (off[i] * group + i (R - 1)) / R on, of each KV head: room for its
// ceil(n * group / R) tiles before the next slice's begin, whatever the offsets are.
constexpr int kCluster = 8;

template <int R>
__device__ __forceinline__ bool paged_locate_item(const PagedArgs &a, int item, PagedCursor<R> &cur) {
    const int lane = threadIdx.x & 31;
    const uint32_t y = (uint32_t)item / (uint32_t)a.hkv;
    auto first = [&](int i) {
        const uint32_t o = (uint32_t)min(max(__ldg(a.off + i), 0), (int32_t)a.nq);
        return (o * (uint32_t)a.group + (uint32_t)i * (R - 1)) / R;
    };
    int count = 0;
    for (int base = 0; base < a.slices; base += 32) {
        const bool before = base + lane < a.slices && first(base + lane) <= y;
        const uint32_t m = __ballot_sync(0xffffffffu, before);
        count += __popc(m);
        if (m != 0xffffffffu) break;
    }
    if (count == 0) return false;
    cur.slice = count - 1;
    cur.s = paged_slice<R>(a, cur.slice);
    cur.g = (int32_t)((uint32_t)item - y * (uint32_t)a.hkv);
    cur.t = y - first(cur.slice);
    cur.start = 0;
    return cur.t < cur.s.tiles;
}

// What the warps of a block need to know of the item they are at: written by the warp that
// walks the row of items (and loads their pages), a few items ahead, so that the others
// neither hold a cursor in registers nor wait for the loads of the next slice.
constexpr int kItemRing = 4;

struct PagedItem {
    int32_t p0, p1;       // pages, p0 < 0: there are no more items
    int32_t row;          // of q, the slice's first
    int32_t token, head;  // the tile's first packed row: token of the slice, head of the group
    int32_t left;         // packed rows from there to the slice's end (at most `rows`)
    int32_t g;            // KV head
    int32_t kb, ke, back; // keys [kb, ke); the causal rule: row `token` sees j < token + back too
    int32_t whole, part;  // all of its pages are here; else the slot for this piece

    // First key that a packed row of the tile does not see.
    __device__ __forceinline__ int32_t limit(int r, int group) const {
        // unsigned: rows behind the last wrap around
        return min(ke, (int32_t)((uint32_t)token + (uint32_t)(head + r) / (uint32_t)group + (uint32_t)back));
    }
};

template <int R>
__device__ __forceinline__ void paged_item(const PagedArgs &a, const PagedCursor<R> &cur, int c, uint32_t lo,
                                           uint32_t hi, PagedItem &x) {
    cur.pages(a, lo, hi, x.p0, x.p1);
    const uint32_t first = cur.t * R;
    x.row = cur.s.r0;
    x.token = (int32_t)(first / (uint32_t)a.group);
    x.head = (int32_t)(first - (uint32_t)x.token * (uint32_t)a.group);
    x.left = (int32_t)min((uint32_t)cur.s.n * (uint32_t)a.group - first, (uint32_t)R);
    x.g = cur.g;
    x.kb = cur.s.kb;
    x.ke = cur.s.ke;
    // token + back <= end and >= -2^31, and without the causal rule never below ke
    x.back = a.causal ? cur.s.end - (cur.s.n - 1) : INT32_MAX - cur.s.n;
    x.whole = lo <= cur.start && cur.end() <= hi;
    x.part = 2 * c + (lo <= cur.start ? 1 : 0);  // odd: begun here
}

// An item begun in share c and ended in share `last` (last < c: there is none).
struct PagedJoin {
    int32_t last;
    int32_t row, token, head, left, g;  // as in PagedItem
    int32_t unused[2];
};
static_assert(sizeof(PagedJoin) == kPagedJoinBytes, "workspace layout");

// What the joining kernel has to know of share c, whose last item is `cur`; one thread.
template <int R>
__device__ __forceinline__ void paged_join_of(const PagedArgs &a, const PagedCursor<R> &cur, const PagedItem &x, int c,
                                              uint32_t hi, uint32_t total) {
    PagedJoin j = {-1, x.row, x.token, x.head, x.left, x.g, {0, 0}};
    if (cur.end() > hi && !(x.part & 1)) j.last = -1;      // it was begun earlier
    else if (cur.end() > hi) {
        // the last share that begins before the item ends: an estimate, put right
        const uint32_t end = cur.end();
        int k = min((int)((float)end / (float)total * paged_shares(R)), paged_shares(R) - 1);
        while (k > c && paged_share<R>(total, k) >= end) --k;
        while (k + 1 < paged_shares(R) && paged_share<R>(total, k + 1) < end) ++k;
        j.last = k;
    }
    a.joins[c] = j;
}

__device__ __forceinline__ float *paged_part(const PagedArgs &a, int d, int slot) {
    return a.part + (size_t)slot * a.rows * (d + 2);
}

// ------------------------------------------------------------------ types

template <typename T>
struct Io;
template <>
struct Io<__nv_bfloat16> {
    static constexpr bool kF16 = false;
    // P = 2^(s - reference) in bf16 has fp32's exponents: no shift is needed
    static constexpr float kShift = 0.f;
    // sums of weights may reach this before the reference moves: fp32's 2^128 leaves room for
    // values up to 2^90 and a hundred thousand keys
    static constexpr float kTop = 1048576.f;  // 2^20
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return sm100::pack_bf16x2(lo, hi); }
    static __device__ __forceinline__ bool bad(uint32_t bits) { return (bits & 0x7f80u) == 0x7f80u; }
    // sum + 0 v in both halves: +-0 as long as every v was finite
    static __device__ __forceinline__ uint32_t add_zero_times(uint32_t v, uint32_t sum) {
        const __nv_bfloat162 r = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&v), __floats2bfloat162_rn(0.f, 0.f),
                                         *reinterpret_cast<const __nv_bfloat162 *>(&sum));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
};
template <>
struct Io<__half> {
    static constexpr bool kF16 = true;
    // The reference is put 6 below the running maximum: P then lies between 2^-24 (fp16's
    // smallest) and 2^6, and before the reference moves up to 2^14 in the few-row kernel (kLazy)
    // and 2^15 in the many-row one (kTop), below fp16's 65504; without it a key 2^-14 below the
    // largest would already lose bits of its P.
    static constexpr float kShift = 6.f;
    static constexpr float kTop = 32768.f;  // no weight above 2^15, below fp16's 65504
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&u));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi) { return sm100::pack_f16x2(lo, hi); }
    static __device__ __forceinline__ bool bad(uint32_t bits) { return (bits & 0x7c00u) == 0x7c00u; }
    static __device__ __forceinline__ uint32_t add_zero_times(uint32_t v, uint32_t sum) {
        const __half2 r = __hfma2(*reinterpret_cast<const __half2 *>(&v), __floats2half2_rn(0.f, 0.f),
                                  *reinterpret_cast<const __half2 *>(&sum));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
};

// The reference moves when a score passes it by more than this (in powers of two).
constexpr float kLazy = 8.f;

// ------------------------------------------------------------------ rows at explicit positions

// cos and sin of position * base^(-i/P).  A whole number of positions times the turns a position
// (in units of 2^-64) modulo 2^64 is the fraction of a turn, exactly but for the turns' own
// rounding, however far the position is (in fp32 position 10^6 would be off by 0.06 rad); its
// upper 32 bits go on to fp32.
__device__ __forceinline__ int32_t paged_turn(int32_t position, uint64_t turns) {
    const uint32_t p = (uint32_t)position, low = (uint32_t)turns, high = (uint32_t)(turns >> 32);
    return (int32_t)(__umulhi(p, low) + p * high - (position < 0 ? low : 0u));  // in units of 2^-32
}
__device__ __forceinline__ float2 paged_cos_sin(int32_t position, uint64_t turns) {
    float2 cs;
    sincospif((float)paged_turn(position, turns) * 4.656612873077393e-10f, &cs.y, &cs.x);  // half turns: 2^-31
    return cs;
}
// The same from the special-function unit, for queries, to 2^-20.5 of the pair's length each: the
// queries of an item are 9,216 angles that stand before its first score (sincospif took 6 us of
// every block's life).  With bf16 values the query is then rounded to fp16, half a step 2^-11, and
// the angle's error does not show.  With fp16 values, whose queries keep what that rounding leaves,
// it is the largest error of a score, 2^-19.6 of |q||k| / sqrt(D); at the norms that QK-Norm gives
// (sqrt(D) each, D = 48) that moves a weight by 9e-6 of itself, beside the 2^-11 by which its own
// rounding to fp16 may.
__device__ __forceinline__ float2 paged_cos_sin_fast(int32_t position, uint64_t turns) {
    const float x = (float)paged_turn(position, turns) * 1.4629180792671596e-9f;  // radians: 2 pi 2^-32
    return make_float2(__cosf(x), __sinf(x));
}

// What eight lanes make of a row: lane e has channel pairs e, e + 8, e + 16 (those below
// D / 2).
template <int D>
struct Row8 {
    static constexpr int P = Geo<D>::PAIRS;
    static constexpr int N = (D / 2 + 7) / 8;
    float2 x[N];
    int32_t at[N];

    // The raw values and the positions, on the way at the same time.  pos: any three words that
    // may be read where there are no positions.
    template <typename T>
    __device__ __forceinline__ void load(const T *row, const int32_t *pos, int e) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int p = min(e + 8 * i, D / 2 - 1);  // lanes without a pair read the last one again
            x[i] = Io<T>::unpack(__ldg(reinterpret_cast<const uint32_t *>(row) + p));
            if (e + 8 * i >= D / 2) x[i] = make_float2(0.f, 0.f);
            at[i] = __ldg(pos + min(p / P, 2));
        }
    }
    // The lane's part of the QK-Norm gain.
    static __device__ __forceinline__ void load_gain(const float *gain, int e, float2 (&gn)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) gn[i] = make_float2(1.f, 1.f);
        if (gain == nullptr) return;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int p = min(e + 8 * i, D / 2 - 1);
            gn[i] = make_float2(__ldg(gain + 2 * p), __ldg(gain + 2 * p + 1));
        }
    }
    // QK-Norm and RoPE.
    __device__ __forceinline__ void prologue(const float2 (&gn)[N], const uint64_t *turns, float eps, int e) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) ss = fmaf(x[i].x, x[i].x, fmaf(x[i].y, x[i].y, ss));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float r = rsqrtf(ss * (1.0f / D) + eps);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int p = e + 8 * i;
            const float y0 = x[i].x * r * gn[i].x, y1 = x[i].y * r * gn[i].y;
            x[i] = make_float2(y0, y1);
            if (p < 3 * P) {
                const float2 cs = paged_cos_sin_fast(at[i], turns[8 * (p / P) + p % P]);
                x[i] = make_float2(y0 * cs.x - y1 * cs.y, y0 * cs.y + y1 * cs.x);
            }
        }
    }
};

// ------------------------------------------------------------------ bounded waits

constexpr uint64_t kPagedWaitNs = 2000000000ull;  // a healthy wait is microseconds

// A thread that finds the phase incomplete asks to be put to sleep for up to 20 us at a time:
// two warps that poll take issue slots from the softmax warps beside them (2 % of paged_tiles).
__device__ __forceinline__ bool paged_wait(uint32_t bar, uint32_t parity, const PagedArgs &a,
                                           volatile int *abort_flag) {
    if (sm100::mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
    const uint64_t t0 = sm100::globaltimer_ns();
    do {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(bar), "r"(parity), "r"(20000u)
            : "memory");
        if (done) return true;
    } while (sm100::globaltimer_ns() - t0 < a.timeout_ns);
    atomicOr(a.status, kPagedTimeout);
    *abort_flag = 1;
    return false;
}

// The warp that walks the items of share c (CL > 1: that has item c / CL, part c % CL): publishes each and moves its pages into the ring, a page's
// keys and values by one bulk copy each, until the block's stretch ends; then waits for the
// copies that are still in flight.  Barriers: full / empty of the STAGES page stages (base +
// 8 i, base + 8 (STAGES + i)), and of the kItemRing items behind them.  here[i]: stage i holds
// a page; an absent one holds no keys.
template <int R, int STAGES, int TILE, int KSTAGE, int STAGE, int CL = 1>
__device__ __forceinline__ void paged_fill(const PagedArgs &a, int c, uint32_t ring, uint32_t bars, uint32_t item_bars, PagedItem *items,
                                           volatile int *here, volatile int *abort_flag) {
    const int lane = threadIdx.x & 31;
    auto full = [&](int i) -> uint32_t { return bars + 8u * (uint32_t)i; };
    auto empty = [&](int i) -> uint32_t { return bars + 8u * (uint32_t)(STAGES + i); };
    constexpr int D = TILE / (2 * kPage);
    PagedCursor<R> cur;
    uint32_t lo, hi, total;
    int it = 0;
    bool more;
    if constexpr (CL > 1) more = paged_locate_item(a, c / CL, cur);
    else more = paged_locate(a, c, lo, hi, total, cur);
    if (CL == 1 && !more) {
        // an empty stretch inside an item that others share: a piece without keys
        if (lane == 0) a.joins[c].last = -1;
        for (int r = lane; r < R; r += 32) {
            paged_part(a, D, 2 * c)[R * D + r] = -INFINITY;
            paged_part(a, D, 2 * c)[R * (D + 1) + r] = 0.f;
        }
    }
    // An item is published when the ring's worth of pages of the one before it is on the way, so
    // that no page waits for it; for the 384-row tiles before those pages, since two warps need the
    // time of four pages for its queries (ragged chunks: 341 us the other way, 318 us).
    constexpr bool kEarly = R >= kPagedNarrowRows;
    int published = 0;
    PagedItem x;
    const int32_t *row = nullptr;
    auto publish = [&] {
        const int slot = published % kItemRing;
        if (published >= kItemRing &&
            !__all_sync(0xffffffffu, paged_wait(item_bars + 8u * (uint32_t)(kItemRing + slot),
                                                (published / kItemRing - 1) & 1, a, abort_flag)))
            return false;
        if (more) {
            if constexpr (CL > 1) {
                paged_item(a, cur, 0, 0, cur.end(), x);
                const int32_t np = x.p1 - x.p0, rank = c % CL;
                x.p1 = x.p0 + (int32_t)((int64_t)np * (rank + 1) / CL);
                x.p0 += (int32_t)((int64_t)np * rank / CL);
            } else {
                paged_item(a, cur, c, lo, hi, x);
            }
            row = a.table + (int64_t)cur.s.b * a.width;
        } else {
            x.p0 = -1;
        }
        if (lane == 0) {
            items[slot] = x;
            sm100::mbar_arrive(item_bars + 8u * (uint32_t)slot);
        }
        ++published;
        return true;
    };
    bool ok = publish();
    while (ok && more) {
        const int32_t p0 = x.p0, p1 = x.p1, g = x.g;
        const int32_t *pages = row;
        const int32_t ahead = kEarly ? p0 : p0 + min(p1 - p0, STAGES);
        auto next = [&] {
            if constexpr (CL > 1) {
                more = false;
            } else {
                if (lane == 0 && cur.end() >= hi) paged_join_of(a, cur, x, c, hi, total);
                more = cur.end() < hi && cur.next(a);
            }
            return publish();
        };
        if (ahead == p0) ok = next();
        for (int32_t base = p0; base < p1 && ok; base += 32) {
            const int32_t mine = base + lane < p1 ? __ldg(pages + base + lane) : -1;
            const int count = min(32, p1 - base);
            for (int j = 0; j < count; ++j) {
                const int32_t page = __shfl_sync(0xffffffffu, mine, j);
                if (lane == 0 && ok && !a.skip_loads) {
                    const int st = it % STAGES;
                    if (it >= STAGES) ok = paged_wait(empty(st), (it / STAGES - 1) & 1, a, abort_flag);
                    if (ok) {
                        const bool on = page >= 0 && page < a.pages;
                        here[st] = on;
                        if (on) {
                            const int64_t at = ((int64_t)page * a.hkv + g) * TILE;
                            const uint32_t dst = ring + st * STAGE;
                            sm100::mbar_arrive_expect_tx(full(st), 2 * TILE);
                            sm100::bulk_g2s(dst, static_cast<const uint8_t *>(a.k_pages) + at, TILE, full(st));
                            sm100::bulk_g2s(dst + KSTAGE, static_cast<const uint8_t *>(a.v_pages) + at, TILE, full(st));
                        } else {
                            sm100::mbar_arrive(full(st));
                        }
                        ++it;
                    }
                }
                if (!kEarly && base + j + 1 == ahead) {
                    ok = __shfl_sync(0xffffffffu, ok, 0);
                    if (ok) ok = next();
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
        }
    }
    if (CL == 1 && !ok && lane == 0) a.joins[c].last = -1;
    // every copy must have landed before the block may end
    if (lane == 0)
        for (int j = it > STAGES ? it - STAGES : 0; j < it; ++j)
            if (!sm100::mbar_wait(full(j % STAGES), (j / STAGES) & 1, a.timeout_ns)) {
                atomicOr(a.status, kPagedTimeout);
                *abort_flag = 1;
            }
    __syncwarp();
}

}  // namespace bca
