// The warps' own matrix instructions over page tiles, and what a page's slots that a row does
// not see need: shared by the kernels of paged attention.
#pragma once

#include "paged_device.cuh"

namespace bca {

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm2(uint32_t addr, uint32_t &r0, uint32_t &r1) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0,%1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}

// V of 16 tokens: vf[n] is the B operand of channels 8 n .. 8 n + 7 (lane (g, t): channel g,
// tokens 2 t, 2 t + 1 and 8 more).  addr: the lane's row, token group (lane / 8) % 2, channel
// group lane / 16.
template <int NV>
__device__ __forceinline__ void ldsm_v(uint32_t addr, uint32_t (&vf)[NV][2]) {
#pragma unroll
    for (int n = 0; n + 1 < NV; n += 2) {
        uint32_t r[4];
        ldsm4(addr + n * 128, r);
        vf[n][0] = r[0];
        vf[n][1] = r[1];
        vf[n + 1][0] = r[2];
        vf[n + 1][1] = r[3];
    }
    if constexpr (NV % 2 == 1) ldsm2(addr + (NV - 1) * 128, vf[NV - 1][0], vf[NV - 1][1]);
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

// A weight of 0 does not silence a NaN or an infinity.  So, where some row does not see all of
// the 16 tokens whose V is in vf, values that are not finite are taken out of vf, if there are any
// (0 times a value, summed up, is NaN then): those of tokens that no row sees (outside
// [kb, end)) for good, and true (for the whole warp) if others are left, which add_left_out then
// gives to the rows that do see their token.  key: that of the lane's first token.
template <typename T, int NV>
__device__ __forceinline__ bool clear_unseen(uint32_t (&vf)[NV][2], int32_t key, int32_t kb, int32_t end) {
    uint32_t test[2] = {0u, 0u};
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
        for (int b = 0; b < 2; ++b) test[b] = Io<T>::add_zero_times(vf[n][b], test[b]);
    if (!__any_sync(0xffffffffu, ((test[0] | test[1]) & 0x7fff7fffu) != 0u)) return false;
    bool odd = false;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        const int32_t k = key + 8 * b;
        const uint32_t keep = (k >= kb && k < end ? 0xffffu : 0u) | (k + 1 >= kb && k + 1 < end ? 0xffff0000u : 0u);
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
    return __any_sync(0xffffffffu, odd);
}

// o += p v over the values that clear_unseen left out, for the rows that see their token: p the
// weights as A operand, v the two token groups in shared memory, lim where the lane's two rows'
// keys end.  Rare, so written for size; inlined, since arrays handed to a function that is not
// live in memory.
template <int D, typename T, int NV>
__device__ __forceinline__ void add_left_out(float (&o)[NV][4], const uint32_t (&p)[4], const T *v, int32_t key0,
                                             int32_t kb, const int32_t (&lim)[2]) {
    const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll 1
    for (int x = 0; x < 16; ++x) {
        const int src = (lane & ~3) + (x % 8) / 2;
        float w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 both = Io<T>::unpack(__shfl_sync(0xffffffffu, x < 8 ? p[h] : p[2 + h], src));
            w[h] = x % 2 ? both.y : both.x;
        }
        const int32_t key = key0 + x;
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const T y = v[(x / 8 * D + 8 * n + 2 * t + (j & 1)) * 8 + x % 8];
                if (Io<T>::bad(*reinterpret_cast<const uint16_t *>(&y)) && key >= kb && key < lim[j >> 1])
                    o[n][j] += w[j >> 1] * (float)y;
            }
    }
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

}  // namespace bca
