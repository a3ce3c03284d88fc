// Warp-level building blocks of the gated delta rule's chunked kernels: 64-row bf16 tiles
// in shared memory, the fragments of mma.m16n8k16 read from them, and fp32 values held as
// pairs of bf16.
//
// Tiles.  A tile of 64-column blocks, each [rows][128 bytes] with the 16-byte chunk index
// XORed by (row mod 8): any eight consecutive rows of one chunk column lie in different
// banks, so every ldmatrix below is free of conflicts.
//
// Pairs.  x = hi + lo with hi = bf16(x), lo = bf16(x - hi): |x - hi - lo| <= 2^-16 |x|.
// A product of a pair with an exact bf16 operand is two MMAs, of two pairs three (the
// lo lo term, 2^-16 of the result, is left out).
//
// Three terms, the third bf16 of what the pair leaves, hold x to 2^-24 of itself, as fp32
// does; a product of two such is six MMAs (down to the second order), of one with a pair five.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

namespace wkv7 {
namespace gdr {

constexpr int C = 64;               // tokens per chunk
constexpr uint32_t kTile = C * 128;  // bytes of a 64-row, 64-column block

template <int ROWS>
__device__ __forceinline__ uint32_t tile_off(int row, int col) {
    return static_cast<uint32_t>((col >> 6) * (ROWS * 128) + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4));
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}

// c += A (16 x 16) B (16 x 8).  A: a0 (row g, cols 2q,2q+1), a1 (row g + 8), a2 (cols + 8),
// a3 (row g + 8, cols + 8); B: b0 (rows 2q,2q+1, col g), b1 (rows + 8); C: c0,c1 (row g, cols
// 2q,2q+1), c2,c3 (row g + 8); g = lane / 4, q = lane % 4.
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Fragment loads from a tile of ROWS rows (lane-dependent addresses):
// B for two column tiles n0, n0 + 8 over k0 .. k0 + 15 from a tile [n][k].
template <int ROWS>
__device__ __forceinline__ void load_b(uint32_t tile, int n0, int k0, int lane, uint32_t (&r)[4]) {
    ldsm4(tile + tile_off<ROWS>(n0 + ((lane >> 4) << 3) + (lane & 7), k0 + (lane & 8)), r);
}
// A for rows m0 .. m0 + 15 over k0 .. k0 + 15 from a tile [k][m].
template <int ROWS>
__device__ __forceinline__ void load_at(uint32_t tile, int m0, int k0, int lane, uint32_t (&r)[4]) {
    ldsm4t(tile + tile_off<ROWS>(k0 + ((lane >> 4) << 3) + (lane & 7), m0 + (lane & 8)), r);
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float low(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// (a, b) - (c, d), (a, b) * c and (a c, b d) in one instruction each.
__device__ __forceinline__ void sub2(float &a, float &b, float c, float d) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tsub.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}
__device__ __forceinline__ void mul2(float &a, float &b, float c) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %2};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c));
}

__device__ __forceinline__ void mul2(float &a, float &b, float c, float d) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(c), "f"(d));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {  // a b + c, two at a time
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)),
          "l"(*reinterpret_cast<unsigned long long *>(&c)));
    return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long d;
    asm("mul.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long d;
    asm("add.rn.f32x2 %0, %1, %2;"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 pair(uint32_t u) { return make_float2(low(u), high(u)); }
// 2^x to two units in the last place, and 0 below the normal numbers.
__device__ __forceinline__ float exp2_flush(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two fp32 values as a pair of packed bf16 pairs.
__device__ __forceinline__ void split(float x, float y, uint32_t &hi, uint32_t &lo) {
    hi = pack(x, y);
    sub2(x, y, low(hi), high(hi));
    lo = pack(x, y);
}
// And as three terms.
__device__ __forceinline__ void split3(float x, float y, uint32_t &a, uint32_t &b, uint32_t &c) {
    a = pack(x, y);
    sub2(x, y, low(a), high(a));
    split(x, y, b, c);
}
// The A fragment (16 rows x 16 columns), in three terms, of an accumulator's two neighbouring column tiles.
__device__ __forceinline__ void split_a(const float (&c0)[4], const float (&c1)[4], uint32_t (&x)[3][4]) {
    split3(c0[0], c0[1], x[0][0], x[1][0], x[2][0]);
    split3(c0[2], c0[3], x[0][1], x[1][1], x[2][1]);
    split3(c1[0], c1[1], x[0][2], x[1][2], x[2][2]);
    split3(c1[2], c1[3], x[0][3], x[1][3], x[2][3]);
}

// 16 bytes global -> shared without registers; zeros where `in` is false (src is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in) {
    const int n = in ? 16 : 0;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int K>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(K) : "memory");
}

}  // namespace gdr
}  // namespace wkv7
