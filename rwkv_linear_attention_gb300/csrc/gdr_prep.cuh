// The state-independent part of the gated delta rule's chunked form: per chunk of 64
// tokens and value head, with gam = the running sum of g inside the chunk (inclusive),
//
//   Ahat_ts = e^{gam_t - gam_s} (k_t . k_s) beta_s   (s < t)     That = (I + Ahat)^{-1}
//   P_ts    = scale e^{gam_t - gam_s} (q_t . k_s) beta_s   (s <= t)
//   d_t = e^{gam_t}     e'_s = e^{gam_C - gam_s}     e_s = e'_s beta_s
//
// From u_t = beta_t (v_t - S~_t^T k_t) unrolled over the chunk: with err_t = u_t / beta_t,
//   err = That (V - d K S0),  o = scale d Q S0 + P err,  S_C = d_C S0 + K^T (e err).
// Writing the strength beta into the columns instead of the rows keeps err itself, so
// the gradient needs no division by beta.
//
// The products k_t . k_s and q_t . k_s (exact products of bf16, fp32 sums) are one MMA of the 128
// rows (K, Q) with the 64 rows of K: row t of the first lies in TMEM lane t, of the second in lane
// 64 + t, and the thread of that lane decays it.  Exponents are kept as an integer and a
// fraction of log2, so that a large decay in a chunk costs the others no digits.  Only the
// diagonal blocks take an exponential per element: left of them the decay is a product of two
// factors, both at most 1 where g <= 0, of the row since its block's first token and of the
// column up to it.
//
// The inverse goes by 16 x 16 blocks.  The two warps that hold Ahat's rows invert their diagonal
// blocks in fp32, one column per lane by substitution (stable for any Ahat, unlike its powers),
// while the other two form P.  Then warp j forms the blocks below diagonal block j,
// T_ij = -T_ii sum_{j <= m < i} A_im T_mj, transposed on the tensor cores: T_mj^T is a left
// operand in registers, A_im^T and T_ii^T are right operands read from bf16 tiles
// (gdr_mma.cuh), and no warp waits for another between the blocks of its column.
//
// That and the products that form it are in three bf16 terms, where pairs serve for the rest: with keys that
// repeat and strengths near 2, That's elements stay near 2 all over the chunk and That times a
// vector is a small difference of large terms.  With That in pairs, 1024 tokens of one key of 128 channels
// with strength 2 and no decay came out 3e-2 off; in three terms, 5e-4 (independent keys: 7e-6
// either way).
#pragma once

#include "gdr_internal.cuh"
#include "gdr_tc.cuh"

namespace wkv7 {
namespace gdr {

// The vectors of a chunk, 64 floats each; the first six are kept for the backward.
enum Vec {
    kVecD = 0, kVecE = C, kVecBeta = 2 * C, kVecInt = 3 * C, kVecFrac = 4 * C, kVecE1 = 5 * C, kVecKept = 6 * C,
    kVecRow = 6 * C,           // e^{gam_t - m}, m = the sum before the token's block of 16 (blocks 1 - 3)
    kVecCol = 7 * C,           // e^{m - gam_s} beta_s for the tokens before blocks 1, 2, 3, 48 places each
    kVecFloats = 7 * C + 3 * 48
};

// A number of log2 as integer plus fraction in [-1/2, 1/2].
struct Log2 {
    float i, f;
};
__device__ __forceinline__ Log2 normal(float i, float f) {
    const float r = rintf(f);
    return {i + r, f - r};
}
__device__ __forceinline__ Log2 log2_of_exp(float g) {  // g log2(e), log2(e) = hi + lo
    const float hi = 1.44269502162933349609375f, lo = 1.925962991126617468870e-8f;
    const float i = rintf(g * hi);
    return normal(i, fmaf(g, hi, -i) + g * lo);
}

// One warp: the vectors of tokens t0 .. t1 - 1 (zero strength and no decay behind them).
__device__ __forceinline__ void chunk_vectors(const GdrPrefillArgs &p, int h, int t0, int t1, int lane, float *vec) {
    Log2 x[2];
    float beta[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int t = t0 + 2 * lane + j;
        const bool in = t < t1;
        const long long at = static_cast<long long>(in ? t : t0) * p.Hv + h;
        x[j] = in ? log2_of_exp(gdr_clamp_decay(p.g[at])) : Log2{0.f, 0.f};
        beta[j] = in ? p.beta[at] : 0.f;
    }
    Log2 sum = normal(x[0].i + x[1].i, x[0].f + x[1].f);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float i = __shfl_up_sync(0xffffffffu, sum.i, off), f = __shfl_up_sync(0xffffffffu, sum.f, off);
        if (lane >= off) sum = normal(sum.i + i, sum.f + f);
    }
    const float endi = __shfl_sync(0xffffffffu, sum.i, 31), endf = __shfl_sync(0xffffffffu, sum.f, 31);
    float i = __shfl_up_sync(0xffffffffu, sum.i, 1), f = __shfl_up_sync(0xffffffffu, sum.f, 1);
    if (lane == 0) i = f = 0.f;
    const Log2 first = normal(i + x[0].i, f + x[0].f);
    const Log2 gam[2] = {first, sum};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int t = 2 * lane + j;
        const float e = exp2f((endi - gam[j].i) + (endf - gam[j].f));
        vec[kVecD + t] = exp2f(gam[j].i + gam[j].f);
        vec[kVecE + t] = e * beta[j];
        vec[kVecBeta + t] = beta[j];
        vec[kVecInt + t] = gam[j].i;
        vec[kVecFrac + t] = gam[j].f;
        vec[kVecE1 + t] = e;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 5; ++j) {  // 64 of the rows, then 16 + 32 + 48 of the columns
        const int i = j * 32 + lane, k = i - C;
        const int block = j < 2 ? i >> 4 : k < 16 ? 1 : k < 48 ? 2 : 3;
        const int t = j < 2 ? i : k - (block == 1 ? 0 : block == 2 ? 16 : 48), m = 16 * block - 1;
        if (block == 0) continue;
        const float di = vec[kVecInt + t] - vec[kVecInt + m], df = vec[kVecFrac + t] - vec[kVecFrac + m];
        if (j < 2) vec[kVecRow + t] = exp2f(di + df);
        else vec[kVecCol + (block - 1) * 48 + t] = exp2f(-di - df) * vec[kVecBeta + t];
    }
}

// x or 0, as a selection: a branch around each element's exponential costs more than all of them.
__device__ __forceinline__ float keep(bool c, float x) {
    float r;
    asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\tselp.f32 %0, %1, 0f00000000, p;\n\t}" : "=f"(r) : "f"(x), "r"(static_cast<uint32_t>(c)));
    return r;
}

constexpr int kDiagLd = 20;  // fp32 row stride of a diagonal block

// Four warps (w = 0 .. 3, the TMEM lane quarter each): That and P of a chunk from the products at TMEM
// column `gram`: That's three tiles into shared memory at `t_at`, P hi, lo straight to `p_out`.
// Ahat's block (i, m), i > m, lies meanwhile in That's place for (m, i), which is not That's own.
// `diag`: four blocks of 16 x kDiagLd floats; BAR: a named barrier of these four warps, which they
// have passed since any of the scratch was read.
template <int BAR>
__device__ __forceinline__ void chunk_matrices(unsigned char *smem, uint32_t gram, uint32_t t_at, unsigned char *p_out, float *diag,
                                               const float *vec, float scale, int w, int lane) {
    const uint32_t ttile = ptx::smem_addr(smem) + t_at;
    {
        const int t = (w & 1) * 32 + lane, own = t >> 4;  // this thread's row and its block row
        const bool is_q = w >= 2;
        const float ti = vec[kVecInt + t], tf = vec[kVecFrac + t], mul = is_q ? scale : 1.f;
        const int parts = (w & 1) ? 4 : 2;  // rows 0 - 31 have no more than 32 columns
        const float row = own > 0 ? vec[kVecRow + t] * mul : 0.f;
        const float *colf = vec + kVecCol + (own > 0 ? own - 1 : 0) * 48;
        float y[16];
#pragma unroll 1
        for (int p = 0; p < parts; ++p) {  // the blocks left of the diagonal
            float x[16];
            tm_ld<16>(gram + (static_cast<uint32_t>(w * 32) << 16) + p * 16, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = p <= own ? x[i] : y[i];  // at last the diagonal block
            if (p < own) {
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(colf + p * 16 + i);
                    mul2(x[i], x[i + 1], f.x, f.y);
                    mul2(x[i + 2], x[i + 3], f.z, f.w);
                    mul2(x[i], x[i + 1], row);
                    mul2(x[i + 2], x[i + 3], row);
                }
                if (is_q) {
                    uint32_t hi[8], lo[8];
                    split_row<16>(x, hi, lo);
                    store_row_global<C>(p_out, p_out + kTile, t, p * 16, hi, lo);
                } else {
                    uint32_t x0[8], x1[8], x2[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) split3(x[2 * i], x[2 * i + 1], x0[i], x1[i], x2[i]);
                    unsigned char *at = smem + t_at;
#pragma unroll
                    for (int i = 0; i < 8; i += 4) {
                        const uint32_t off = tile_off<C>(p * 16 + (t & 15), own * 16 + 2 * i);
                        *reinterpret_cast<uint4 *>(at + off) = make_uint4(x0[i], x0[i + 1], x0[i + 2], x0[i + 3]);
                        *reinterpret_cast<uint4 *>(at + off + kTile) = make_uint4(x1[i], x1[i + 1], x1[i + 2], x1[i + 3]);
                        *reinterpret_cast<uint4 *>(at + off + 2 * kTile) = make_uint4(x2[i], x2[i + 1], x2[i + 2], x2[i + 3]);
                    }
                }
            }
        }
        const int last = is_q ? t & 15 : (t & 15) - 1;  // the last column of the diagonal block that counts
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const int s = own * 16 + i;
            const float4 si = *reinterpret_cast<const float4 *>(vec + kVecInt + s);
            const float4 sf = *reinterpret_cast<const float4 *>(vec + kVecFrac + s);
            const float4 be = *reinterpret_cast<const float4 *>(vec + kVecBeta + s);
            const float f0 = exp2_flush((ti - si.x) + (tf - sf.x)) * (be.x * mul), f1 = exp2_flush((ti - si.y) + (tf - sf.y)) * (be.y * mul);
            const float f2 = exp2_flush((ti - si.z) + (tf - sf.z)) * (be.z * mul), f3 = exp2_flush((ti - si.w) + (tf - sf.w)) * (be.w * mul);
            y[i] = keep(i <= last, y[i] * f0);
            y[i + 1] = keep(i + 1 <= last, y[i + 1] * f1);
            y[i + 2] = keep(i + 2 <= last, y[i + 2] * f2);
            y[i + 3] = keep(i + 3 <= last, y[i + 3] * f3);
        }
        if (is_q) {
            uint32_t hi[8], lo[8];
            split_row<16>(y, hi, lo);
            store_row_global<C>(p_out, p_out + kTile, t, own * 16, hi, lo);
        } else {  // Ahat's in fp32
            float *dr = diag + own * 16 * kDiagLd + (t & 15) * kDiagLd;
#pragma unroll
            for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(dr + i) = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
        }
    }
    // the inverses of this warp's two diagonal blocks, one per half warp, lane j holding column j
    if (w < 2) {
        __syncwarp();
        const int j = lane & 15, blk = 2 * w + (lane >> 4);
        const float *dg = diag + blk * 16 * kDiagLd;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float s0 = i == j ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
            for (int m = 0; m < i; m += 4) {
                const float4 a = *reinterpret_cast<const float4 *>(dg + i * kDiagLd + m);
                s0 = fmaf(-a.x, x[m], s0);
                if (m + 1 < i) s1 = fmaf(-a.y, x[m + 1], s1);
                if (m + 2 < i) s0 = fmaf(-a.z, x[m + 2], s0);
                if (m + 3 < i) s1 = fmaf(-a.w, x[m + 3], s1);
            }
            x[i] = s0 + s1;  // exactly 0 above the diagonal
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const __nv_bfloat16 x0 = __float2bfloat16_rn(x[i]);
            const float left = x[i] - __bfloat162float(x0);
            const __nv_bfloat16 x1 = __float2bfloat16_rn(left);
            const uint32_t off = t_at + tile_off<C>(blk * 16 + i, blk * 16 + j) + (j & 7) * 2;
            *reinterpret_cast<__nv_bfloat16 *>(smem + off) = x0;
            *reinterpret_cast<__nv_bfloat16 *>(smem + off + kTile) = x1;
            *reinterpret_cast<__nv_bfloat16 *>(smem + off + 2 * kTile) = __float2bfloat16_rn(left - __bfloat162float(x1));
        }
    }
    ptx::named_sync<BAR, 128>();
    // the blocks below the diagonal: T_mj^T for j = w as left operands
    if (w == 3) return;
    uint32_t t[4][3][4];  // by block row, in three terms
#pragma unroll
    for (int m = 0; m < 3; ++m)
        if (m == w)
#pragma unroll
            for (int x = 0; x < 3; ++x) load_at<C>(ttile + x * kTile, m * 16, m * 16, lane, t[m][x]);
    // d += a times the block at (row, col): the products of terms down to the second order, the smallest first
    auto times = [&](float (&d)[2][4], const uint32_t (&a)[3][4], int row, int col) {
#pragma unroll
        for (int y = 2; y >= 0; --y) {
            uint32_t b[4];
            load_b<C>(ttile + y * kTile, row, col, lane, b);
#pragma unroll
            for (int x = 2 - y; x >= 0; --x)
#pragma unroll
                for (int c = 0; c < 2; ++c) mma(d[c], a[x], b[2 * c], b[2 * c + 1]);
        }
    };
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        if (i <= w) continue;
        float acc[2][4] = {}, res[2][4] = {};
#pragma unroll
        for (int m = 0; m < i; ++m)
            if (m >= w) times(acc, t[m], m * 16, i * 16);  // Ahat_im, in the place for (m, i)
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[c][e] = -acc[c][e];
        uint32_t a[3][4];
        split_a(acc[0], acc[1], a);
        times(res, a, i * 16, i * 16);
        split_a(res[0], res[1], t[i]);
        const uint32_t at = tile_off<C>(i * 16 + ((lane >> 4) << 3) + (lane & 7), w * 16 + (lane & 8));
#pragma unroll
        for (int x = 0; x < 3; ++x) stsm4t(ttile + x * kTile + at, t[i][x][0], t[i][x][1], t[i][x][2], t[i][x][3]);
    }
}

}  // namespace gdr
}  // namespace wkv7
