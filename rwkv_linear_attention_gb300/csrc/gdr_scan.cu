// Token-serial prefill of the gated delta rule (wkv7_gdr_prefill with fp32 inputs), exact
// fp32 throughout, G = 4 or 8 tokens at a time.
//
// With S the state before the G tokens, d_t = prod_{m <= t} e^{g_m}, w_tj = prod_{j < m <= t} e^{g_m}:
//
//   u_t = beta_t (v_t - d_t S^T k_t) - sum_{j < t} beta_t w_tj (k_t . k_j) u_j
//   o_t = scale (d_t S^T q_t + sum_{j <= t} w_tj (q_t . k_j) u_j)
//   S   = d_last S + sum_j k_j (w_last,j u_j)^T
//
// The chain from state to state (a sum over the rows, the solve, the update) bounds the kernel,
// not memory, and one warp's instructions on it (36% of its issue slots filled): token by token
// it took 0.25 us a token at N = 64 and 0.46 at 128; in groups it takes 0.12 and 0.18 in the
// narrowest split.  The products of the inputs (k_t . k_j, q_t . k_j) are off it.
//
// One warp owns 4 kCols columns of one (sequence, head) and keeps that slice of S in registers
// (lane L: kCols columns, rows 4 (L >> 2) + {0 .. 3} of each 32, as pairs of rows for the
// two-wide FMAs).  Four warps of a CTA share a ring of kStages x kTok tokens' vectors in shared
// memory, filled by asynchronous copies; the products for the next kTok tokens are formed while
// these are worked on, by four more warps (the feeders) or by the same.  Tokens behind a
// sequence's last are filled with zeros.
#include "gdr_internal.cuh"
#include "gdr_mma.cuh"
#include "gdr_split.h"
#include "sm103_ptx.cuh"

namespace wkv7 {
namespace {

constexpr int kTok = 16, kStages = 4, kWorkers = 128;

__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool in) {  // zero where `in` is false
    const int n = in ? 4 : 0;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// Two state elements at element index idx, widened; and the rounded store.
__device__ __forceinline__ float2 load_pair(const void *base, wkv7_dtype dt, long long idx) {
    if (dt == WKV7_F32) return *reinterpret_cast<const float2 *>(static_cast<const float *>(base) + idx);
    const uint32_t u = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(base) + idx);
    if (dt == WKV7_BF16) return make_float2(gdr::low(u), gdr::high(u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&u));
}
__device__ __forceinline__ void store_pair(void *base, wkv7_dtype dt, long long idx, float2 x) {
    if (dt == WKV7_F32) {
        *reinterpret_cast<float2 *>(static_cast<float *>(base) + idx) = x;
        return;
    }
    const __half2 f = __floats2half2_rn(x.x, x.y);
    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(base) + idx) =
        dt == WKV7_BF16 ? gdr::pack(x.x, x.y) : *reinterpret_cast<const uint32_t *>(&f);
}

// One level of a sum across lanes that leaves each lane half of its values: the lane gives x[H ..] away and
// keeps x[.. H - 1], plus what the lane `mask` away gives.  The two hold their values in such orders
// that x[H + i] of one is x[i] of the other.
template <int H>
__device__ __forceinline__ void halve(float *x, int mask) {
#pragma unroll
    for (int i = 0; i < H; ++i) x[i] += __shfl_xor_sync(0xffffffffu, x[H + i], mask);
}

// kCols columns a lane and G tokens at a time: 16 sums a lane either way.
template <int N, int kCols, bool kFeeders>
struct Ring {
    static constexpr int G = 16 / kCols;
    static constexpr int kThreads = kFeeders ? 256 : 128;  // with four more warps for the copies and products, or not
    static constexpr int kV = 16 * kCols;                // the CTA's columns
    static constexpr int kQ = kTok * N, kVAt = 2 * kTok * N, kG = kVAt + kTok * kV, kB = kG + kTok;
    static constexpr int kFloats = kB + kTok;
    // What G tokens need besides their vectors: beta w (k . k) [t][j], scale w (q . k) [t][j], beta,
    // beta d, the decay behind each token, scale d, and d of the last.
    static constexpr int kKk = 0, kQk = G * G, kBeta = 2 * G * G, kBetaD = kBeta + G, kBehind = kBetaD + G, kScaleD = kBehind + G,
                         kAll = kScaleD + G, kCoef = kAll + 4;
    static constexpr int kCoefAt = kStages * kFloats;    // of two blocks
    static constexpr int kSumAt = kCoefAt + 2 * (kTok / G) * kCoef;  // per warp: two [token][column] sums
    static constexpr int kBytes = (kSumAt + 4 * 2 * 64) * 4;
};

template <int N, int kCols, bool kFeeders>
__global__ void __launch_bounds__(Ring<N, kCols, kFeeders>::kThreads, 1)
wkv7_gdr_prefill_scan_kernel(const GdrPrefillArgs p) {
    using Rg = Ring<N, kCols, kFeeders>;
    constexpr int R = N / 8, G = Rg::G;
    extern __shared__ __align__(16) float ring[];
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
    const bool feeds = !kFeeders || threadIdx.x >= kWorkers, works = threadIdx.x < kWorkers;
    const int tid = threadIdx.x & (kWorkers - 1);  // among those that feed
    constexpr int kParts = N / Rg::kV;
    const int part = blockIdx.x % kParts, h = blockIdx.x / kParts % p.Hv, hk = h / (p.Hv / p.Hk);
    const int b = gdr_by_length(p.cu_seqlens, p.num_seqs, blockIdx.x / kParts / p.Hv, lane);
    // The sums over the rows leave the lane with one token of G and one pair of columns: its own.  It
    // holds the tokens' sums and its pairs of columns in the order that puts its own first.
    const int own = G == 8 ? ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1) : ((lane >> 4) & 1) * 2 + ((lane >> 3) & 1);
    const int flip = G == 8 ? 0 : ((lane >> 2) & 1) * 2;
    const int col0 = part * Rg::kV, in_warp = (lane & 3) * kCols, mine = warp * 4 * kCols + in_warp;
    const int row0 = (lane >> 2) * 4;  // and + 32, ...
    int bos, eos;
    if (!gdr_seq_bounds(p.cu_seqlens, p.num_seqs, p.T_total, b, bos, eos)) {
        if (threadIdx.x == 0 && h == 0 && part == 0) report(p.status, kDevBadSeqlens);
        return;
    }
    const int blocks = (eos - bos + kTok - 1) / kTok;
    auto load = [&](int i) {  // the tokens of block i; an empty group behind the last, to keep the count
        if (i < blocks) {
            const int t0 = bos + i * kTok, n = min(kTok, eos - t0), rows = (n + G - 1) / G * G;
            float *dst = ring + (i % kStages) * Rg::kFloats;
            for (int e = tid; e < rows * (N / 4); e += kWorkers) {
                const int t = e / (N / 4), c = (e % (N / 4)) * 4;
                const bool in = t < n;
                const long long qk = (static_cast<long long>(in ? t0 + t : t0) * p.Hk + hk) * N + c;
                gdr::copy16(ptx::smem_addr(dst + t * N + c), static_cast<const float *>(p.k) + qk, in);
                gdr::copy16(ptx::smem_addr(dst + Rg::kQ + t * N + c), static_cast<const float *>(p.q) + qk, in);
            }
            for (int e = tid; e < rows * (Rg::kV / 4); e += kWorkers) {
                const int t = e / (Rg::kV / 4), c = (e % (Rg::kV / 4)) * 4;
                const bool in = t < n;
                const long long v = (static_cast<long long>(in ? t0 + t : t0) * p.Hv + h) * N + col0 + c;
                gdr::copy16(ptx::smem_addr(dst + Rg::kVAt + t * Rg::kV + c), static_cast<const float *>(p.v) + v, in);
            }
            if (tid < rows) {
                const bool in = tid < n;
                const long long at = static_cast<long long>(in ? t0 + tid : t0) * p.Hv + h;
                copy4(ptx::smem_addr(dst + Rg::kG + tid), p.g + at, in);
                copy4(ptx::smem_addr(dst + Rg::kB + tid), p.beta + at, in);
            }
        }
        gdr::copy_commit();
    };
    // The coefficients of tokens 4 warp .. + 3 of block i with all tokens of their group: lane L sums
    // the products of token L & 3 over its rows, and is left with G / 4 of them.
    auto products = [&](int i) {
        const int g0 = warp * 4 / G * G;  // the group's first token
        if (i >= blocks || bos + i * kTok + g0 >= eos) return;
        const float *st = ring + (i % kStages) * Rg::kFloats;
        float *cf = ring + Rg::kCoefAt + ((i & 1) * (kTok / G) + g0 / G) * Rg::kCoef;
        const int t = warp * 4 - g0 + (lane & 3);
        const bool q_half = lane & 16;  // left with q . k, else k . k; and with tokens 4, 2, 1 (from the other two bits) on
        const int first = G == 8 ? (lane & 8 ? 4 : 0) + (lane & 4 ? 2 : 0) : (lane & 8 ? 2 : 0) + (lane & 4 ? 1 : 0);
        const float *at = st + (g0 + t) * N + row0, *kj = st + g0 * N + row0;
        float2 s2[2][G] = {};
#pragma unroll
        for (int r = 0; r < N; r += 32) {
            const float4 a = *reinterpret_cast<const float4 *>(at + (q_half ? Rg::kQ : 0) + r);
            const float4 c = *reinterpret_cast<const float4 *>(at + (q_half ? 0 : Rg::kQ) + r);
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const float4 k = *reinterpret_cast<const float4 *>(kj + (j ^ first) * N + r);
                s2[0][j] = gdr::fma2(make_float2(a.z, a.w), make_float2(k.z, k.w), gdr::fma2(make_float2(a.x, a.y), make_float2(k.x, k.y), s2[0][j]));
                s2[1][j] = gdr::fma2(make_float2(c.z, c.w), make_float2(k.z, k.w), gdr::fma2(make_float2(c.x, c.y), make_float2(k.x, k.y), s2[1][j]));
            }
        }
        float s[2 * G];
#pragma unroll
        for (int j = 0; j < 2 * G; ++j) s[j] = s2[j / G][j % G].x + s2[j / G][j % G].y;
        halve<G>(s, 16);
        halve<G / 2>(s, 8);
        halve<G / 4>(s, 4);
        float a[G], upto = 1.f, behind = 1.f;
#pragma unroll
        for (int m = 0; m < G; ++m) {
            a[m] = expf(st[Rg::kG + g0 + m]);
            if (m <= t) upto *= a[m];
            else behind *= a[m];
        }
        const float beta = st[Rg::kB + g0 + t];
#pragma unroll
        for (int e = 0; e < G / 4; ++e) {
            const int j = first + e;
            float w = q_half ? p.scale : beta;
#pragma unroll
            for (int m = 1; m < G; ++m)
                if (m > j && m <= t) w *= a[m];
            cf[(q_half ? Rg::kQk : Rg::kKk) + t * G + j] = (q_half ? j <= t : j < t) ? w * s[e] : 0.f;
        }
        if (lane < 4) {
            cf[Rg::kBeta + t] = beta;
            cf[Rg::kBetaD + t] = beta * upto;
            cf[Rg::kBehind + t] = behind;
            cf[Rg::kScaleD + t] = p.scale * upto;
            if (t == G - 1) cf[Rg::kAll] = upto;
        }
    };

    if (feeds)
        for (int i = 0; i < kStages - 1; ++i) load(i);
    const long long s_at = (static_cast<long long>(b) * p.Hv + h) * (N * N) + col0 + mine;
    auto place = [&](int m, int c) { return s_at + ((m >> 2) * 32 + row0 + (m & 3)) * N + (c ^ flip); };
    float2 x[R / 2][kCols];  // rows in pairs
#pragma unroll
    for (int m = 0; m < R; m += 2)
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
            float2 s0 = make_float2(0.f, 0.f), s1 = s0;
            if (p.initial_state && works) {
                s0 = load_pair(p.initial_state, p.state_dtype, place(m, c));
                s1 = load_pair(p.initial_state, p.state_dtype, place(m + 1, c));
            }
            x[m / 2][c] = make_float2(s0.x, s1.x);
            x[m / 2][c + 1] = make_float2(s0.y, s1.y);
        }
    gdr::copy_wait<kStages - 2>();
    __syncthreads();
    if (feeds) products(0);

    int other[G];  // the lane's order of a group's rows
#pragma unroll
    for (int t = 0; t < G; ++t) other[t] = (t ^ own) * N + row0;
    // the tokens' k or q with the state's columns over the lane's rows; and over all rows, of its own token and pair
    auto dots = [&](const float *rows, float (&s)[16]) {
        float2 z[G][kCols];
#pragma unroll
        for (int r = 0; r < R / 4; ++r)
#pragma unroll
            for (int t = 0; t < G; ++t) {
                const float4 a = *reinterpret_cast<const float4 *>(rows + other[t] + r * 32);
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    const float2 lo = make_float2(a.x, a.y);
                    z[t][c] = r ? gdr::fma2(lo, x[2 * r][c], z[t][c]) : gdr::mul2(lo, x[0][c]);
                }
#pragma unroll
                for (int c = 0; c < kCols; ++c) z[t][c] = gdr::fma2(make_float2(a.z, a.w), x[2 * r + 1][c], z[t][c]);
            }
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = z[e / kCols][e % kCols].x + z[e / kCols][e % kCols].y;
    };
    auto sum = [&](float (&s)[16]) {
        halve<8>(s, 16);
        halve<4>(s, 8);
        halve<2>(s, 4);
    };
    for (int i = 0; i < blocks; ++i) {
        gdr::copy_wait<kStages - 3>();
        __syncthreads();  // block i + 1 has landed, block i's coefficients are written, block i - 1's place is free
        if (feeds) {
            load(i + kStages - 1);
            products(i + 1);
        }
        if (!works) continue;
        const float *st = ring + (i % kStages) * Rg::kFloats;
        const int t0 = bos + i * kTok, n = min(kTok, eos - t0);
#pragma unroll 1
        for (int g = 0; g < n; g += G) {
            const float *kt = st + g * N, *vt = st + Rg::kVAt + g * Rg::kV + mine;
            const float *cf = ring + Rg::kCoefAt + ((i & 1) * (kTok / G) + g / G) * Rg::kCoef;
            float *sums = ring + Rg::kSumAt + (warp * 2 + ((g / G) & 1)) * 64 + in_warp;
            float z[16], y[16];
            dots(kt, z);
            sum(z);
            *reinterpret_cast<float2 *>(sums + own * 4 * kCols + flip) = make_float2(z[0], z[1]);
            dots(kt + Rg::kQ, y);
            __syncwarp();
            auto four = [&](int at) { return *reinterpret_cast<const float4 *>(cf + at); };
            auto pick = [](float4 v, int e) { return e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w; };
            float u[G][kCols];
#pragma unroll
            for (int t = 0; t < G; ++t) {
                const float beta = pick(four(Rg::kBeta + (t & ~3)), t & 3), bd = pick(four(Rg::kBetaD + (t & ~3)), t & 3);
#pragma unroll
                for (int c = 0; c < kCols; c += 2) {
                    const float2 v = *reinterpret_cast<const float2 *>(vt + t * Rg::kV + (c ^ flip));
                    const float2 sk = *reinterpret_cast<const float2 *>(sums + t * 4 * kCols + (c ^ flip));
                    u[t][c] = fmaf(-bd, sk.x, beta * v.x);
                    u[t][c + 1] = fmaf(-bd, sk.y, beta * v.y);
                }
#pragma unroll
                for (int j = 0; j < t; ++j) {
                    const float w = pick(four(Rg::kKk + t * G + (j & ~3)), j & 3);
#pragma unroll
                    for (int c = 0; c < kCols; ++c) u[t][c] = fmaf(-w, u[j][c], u[t][c]);
                }
                if (g + t >= n)
#pragma unroll
                    for (int c = 0; c < kCols; ++c) u[t][c] = 0.f;
            }
            const float2 all = make_float2(cf[Rg::kAll], cf[Rg::kAll]);
#pragma unroll
            for (int m = 0; m < R / 2; ++m)
#pragma unroll
                for (int c = 0; c < kCols; ++c) x[m][c] = gdr::mul2(all, x[m][c]);
#pragma unroll
            for (int t = 0; t < G; ++t) {
                const float behind = pick(four(Rg::kBehind + (t & ~3)), t & 3);
                float2 eu[kCols];
#pragma unroll
                for (int c = 0; c < kCols; ++c) eu[c] = make_float2(behind * u[t][c], behind * u[t][c]);
#pragma unroll
                for (int r = 0; r < R / 4; ++r) {
                    const float4 k = *reinterpret_cast<const float4 *>(kt + t * N + row0 + r * 32);
#pragma unroll
                    for (int c = 0; c < kCols; ++c) {
                        x[2 * r][c] = gdr::fma2(make_float2(k.x, k.y), eu[c], x[2 * r][c]);
                        x[2 * r + 1][c] = gdr::fma2(make_float2(k.z, k.w), eu[c], x[2 * r + 1][c]);
                    }
                }
            }
            sum(y);
            const float sd = cf[Rg::kScaleD + own];
            float2 o = make_float2(sd * y[0], sd * y[1]);
#pragma unroll
            for (int j = 0; j < G; ++j) {
                const float w = pick(four(Rg::kQk + own * G + (j & ~3)), j & 3);
                o.x = fmaf(w, j <= own ? u[j][0] : 0.f, o.x);
                o.y = fmaf(w, j <= own ? u[j][1] : 0.f, o.y);
            }
            if (g + own < n) {
                const long long at = (static_cast<long long>(t0 + g + own) * p.Hv + h) * N + col0 + mine + flip;
                if (p.o_dtype == WKV7_F32) *reinterpret_cast<float2 *>(static_cast<float *>(p.o) + at) = o;
                else *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.o) + at) = gdr::pack(o.x, o.y);
            }
        }
    }
    gdr::copy_wait<0>();
    if (p.final_state && works) {
#pragma unroll
        for (int m = 0; m < R; m += 2)
#pragma unroll
            for (int c = 0; c < kCols; c += 2) {
                store_pair(p.final_state, p.state_dtype, place(m, c), make_float2(x[m / 2][c].x, x[m / 2][c + 1].x));
                store_pair(p.final_state, p.state_dtype, place(m + 1, c), make_float2(x[m / 2][c].y, x[m / 2][c + 1].y));
            }
    }
}

template <int N, int kCols, bool kFeeders>
cudaError_t run(const GdrPrefillArgs &p, cudaStream_t stream) {
    using Rg = Ring<N, kCols, kFeeders>;
    static std::atomic<unsigned long long> allowed{0};
    const cudaError_t e =
        gdr_allow_smem(reinterpret_cast<const void *>(wkv7_gdr_prefill_scan_kernel<N, kCols, kFeeders>), Rg::kBytes, allowed);
    if (e != cudaSuccess) return e;
    const unsigned grid = static_cast<unsigned>(p.num_seqs) * static_cast<unsigned>(p.Hv) * (N / Rg::kV);
    wkv7_gdr_prefill_scan_kernel<N, kCols, kFeeders><<<grid, Rg::kThreads, Rg::kBytes, stream>>>(p);
    return cudaGetLastError();
}

template <int N>
cudaError_t prefill(const GdrPrefillArgs &p, cudaStream_t stream) {
    const GdrSplit s = gdr_choose_split(p.num_seqs, p.T_total, p.Hv, N, p.cu_seqlens_host);
    return s == kGdrNarrow ? run<N, 2, true>(p, stream) : s == kGdrWide ? run<N, 4, true>(p, stream) : run<N, 4, false>(p, stream);
}

}  // namespace

cudaError_t launch_gdr_prefill_scan(const GdrPrefillArgs &p, cudaStream_t s) {
    return p.N == 64 ? prefill<64>(p, s) : prefill<128>(p, s);
}

}  // namespace wkv7
