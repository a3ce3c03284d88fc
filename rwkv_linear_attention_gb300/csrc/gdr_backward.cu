// Gradients of the gated delta rule's prefill (wkv7_gdr_prefill_backward), bf16 inputs.
//
// Per chunk, with That, P, d, e as in gdr_prep.cu (beta in the columns), kk = K K^T, qk =
// Q K^T, w_ts = e^{gam_t - gam_s}, S0 the state before the chunk, G the adjoint of the state
// behind it, do' = scale dO:
//
//   b_s  = e_s (K G)_s + (P^T dO)_s             the adjoint of err
//   dv   = That^T b
//   G0   = d_C G + Q^T (d do') - K^T (d dv)      the adjoint of S0
//   X_ts = do'_t . err_s (s <= t)      M_ts = dv_t . err_s (s < t)
//   dq   = d (do' S0^T) + D K                    D_ts =  beta_s w_ts X_ts
//   dk   = D^T Q + (E + E^T) K - d (dv S0^T) + e Z   E_ts = -beta_s w_ts M_ts,  Z = err G^T
//   dbeta_s = sum_t (w qk X - w kk M)_ts + e'_s k_s . Z_s        (e' = e / beta, kept apart)
//   dgam_t  = sum_s beta_s (w qk X - w kk M)_ts + d_t (q_t . (S0 do'_t) - k_t . (S0 dv_t)) - beta_t dbeta_t
//   dgam_C += sum_s e_s k_s . Z_s + d_C <G, S0> ;  dg = the sums of dgam from each token to its chunk's end
//
// After gdr_prep: the forward chain again (gdr_chain.cuh), keeping S0 and err, and beside it the
// reverse chain below, keeping G and dv; then one CTA per (chunk, query/key head) for the rest, which
// sums the value heads that share the head in a fixed order (no atomics: the same inputs give the
// same bits).
// Every operand that is not an input is a pair of bf16, That has three terms (gdr_mma.cuh).
#include "gdr_chain.cuh"
#include "gdr_internal.cuh"
#include "gdr_prep.cuh"
#include "gdr_tc.cuh"

namespace wkv7 {
namespace {

using namespace gdr;

// ------------------------------------------------------------------ the reverse chain
//
// The forward chain's scheme: one CTA per (sequence, value head), G^T in tensor
// memory, its rows the value columns.  Per chunk, from the last:
//
//   G as pairs (kept), G = d_C G           y = P^T dO (dO across its rows: a left operand in shared memory)
//   x = K G
//   b = e x + y as pairs
//   dv = That^T b                          scale d dO as pairs, where G's pairs were
//   -d dv as pairs                         dv out, and kept as pairs
//   G += Q^T (scale d dO) + K^T (-d dv), the first 64 of its columns before the second
//
// What the chains keep (96 KB each per chunk and head of 128) is more than half of what they move, and
// that bounds them: 466 us together at 4 x 4096 tokens and 32 heads of 128, in which 2.6 GB go through
// HBM (5.5 TB/s).

constexpr uint32_t kMaxPolls = 1u << 17;  // of up to 20 us: seconds

template <int N>
struct Stage {
    static constexpr uint32_t kKQ = 0;                  // K rows 0-63, Q rows 64-127, [128][64] blocks
    static constexpr uint32_t kO = 2 * C * N * 2;       // dO, [64][64] blocks
    static constexpr uint32_t kPrep = kO + C * N * 2;   // P, That, d, e
    static constexpr uint32_t kPrepBytes = kGdrPrepVec + 2 * C * 4;
    static constexpr uint32_t kBytes = kPrep + kGdrPrepVec + 1024;
    static constexpr uint32_t kOutAt = 2 * kBytes;      // dv of one chunk: plain [64][N] bf16, then the low tile
    static constexpr uint32_t kSmem = kOutAt + 2 * C * N * 2;
};

// mbarriers (a stage's own where a waiter could fall a phase behind) and named barriers.
enum Bar { kFull0, kFull1, kDone0, kDone1, kXDone, kDvDone, kG0Done, kG1Done, kBars };
enum Named { kPairs = 1, kAdjoint = 3, kUpdate, kTail, kOutRead, kLast, kOutOnly, kPairsOut, kPairsRead };

template <int N>
__device__ __forceinline__ void reverse_chain(const GdrBackwardArgs &p, const GdrMaps &maps, const unsigned char *__restrict__ prep,
                                              const int32_t *__restrict__ order, const GdrChainStore &keep) {
    using L = Chain<N>;
    using St = Stage<N>;
    constexpr int kColsThreads = L::kWorkers / L::kHalves + 32;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(8) unsigned long long bars[kBars];
    __shared__ uint32_t s_tmem;
    const GdrPrefillArgs &f = p.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x % f.Hv, rank = blockIdx.x / f.Hv;
    const int b = order ? order[rank] : gdr_by_length(f.cu_seqlens, f.num_seqs, rank, lane);
    int bos, eos;
    if (b < 0 || b >= f.num_seqs || !gdr_seq_bounds(f.cu_seqlens, f.num_seqs, f.T_total, b, bos, eos)) return;  // reported by the forward chain
    const long long s_at = (static_cast<long long>(b) * f.Hv + h) * (N * N);
    const int n_chunks = (eos - bos + C - 1) / C;
    if (n_chunks == 0) {  // the adjoint as it was
        ptx::grid_dep_wait();
        if (p.d_initial_state)
            for (int i = threadIdx.x; i < N * N; i += L::kWarps * 32) p.d_initial_state[s_at + i] = p.d_final_state ? p.d_final_state[s_at + i] : 0.f;
        return;
    }
    const uint32_t base = ptx::smem_addr(smem), bar0 = ptx::smem_addr(bars);
    if (warp == L::kMmaWarp) {
        ptx::tmem_alloc(ptx::smem_addr(&s_tmem), 512);
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < kBars; ++i) ptx::mbar_init(bar0 + 8 * i, 1);
            ptx::fence_mbar_init();
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const uint32_t tm = s_tmem;
    const int hk = h / (f.Hv / f.Hk);
    const long long slot0 = (bos >> 6) + b;

    bool dead = false;  // a wait has run out: it is reported, and this thread waits no more
    auto wait = [&](int bar, int phase) {
        if (!dead && !wait_phase(bar0 + 8 * bar, phase & 1, kMaxPolls)) {
            dead = true;
            report(f.status, kDevTimeout);
        }
        ptx::tc_fence_after_sync();
    };
    // everything below counts steps i = 0 ..; step i is chunk n_chunks - 1 - i
    auto wait_full = [&](int i) { wait(kFull0 + (i & 1), i >> 1); };
    auto vec_of = [&](int i) { return reinterpret_cast<const float *>(smem + (i & 1) * St::kBytes + St::kPrep + kGdrPrepVec); };

    if (warp == L::kLoadWarp) {
        if (lane == 0) {
#pragma unroll 1
            for (int i = 0; i < n_chunks; ++i) {
                if (i >= 2) wait(kDone0 + (i & 1), (i - 2) >> 1);  // the stage's chunk is through
                const int c = n_chunks - 1 - i, t0 = bos + c * C;
                const uint32_t s = base + (i & 1) * St::kBytes, full = bar0 + 8 * (kFull0 + (i & 1));
                ptx::mbar_arrive_expect_tx(full, 3 * C * N * 2 + St::kPrepBytes);
#pragma unroll
                for (int j = 0; j < N / 64; ++j) {
                    ptx::tma_load_2d(s + St::kKQ + j * 2 * kTile, &maps.k, hk * N + j * 64, t0, full);
                    ptx::tma_load_2d(s + St::kKQ + j * 2 * kTile + kTile, &maps.q, hk * N + j * 64, t0, full);
                    ptx::tma_load_2d(s + St::kO + j * kTile, &maps.d_o, h * N + j * 64, t0, full);
                }
                ptx::bulk_load(s + St::kPrep, prep + ((slot0 + c) * f.Hv + h) * kGdrPrepBytes, St::kPrepBytes, full);
            }
        }
        return;
    }

    if (warp == L::kMmaWarp) {
        const uint32_t leader = elect_lane();
        constexpr uint32_t kAlong = idesc_bf16(128, 64, false), kAcross = idesc_bf16(128, 64, true);
        constexpr uint32_t kLeftAcross = 1u << 15;  // the left operand too is read across its rows
#pragma unroll 1
        for (int i = 0; i < n_chunks; ++i) {
            const uint32_t s = base + (i & 1) * St::kBytes;
            const uint32_t kq = s + St::kKQ, ot = s + St::kO, ph = s + St::kPrep, th = ph + kGdrPrepThat;
            wait_full(i);
            if (i == 0) ptx::named_sync<kTail, L::kWorkers + 32>();  // rows behind the sequence are zeros
            ptx::tc_fence_after_sync();
            // y: tokens t of block ks reach columns s up to 16 ks + 15 (N = 64: its rows above 63 are not used)
#pragma unroll
            for (int ks = 3; ks >= 0; --ks) {
                const uint32_t id = idesc_bf16(128, 16 * (ks + 1), true) | kLeftAcross;
                const uint64_t ad = sdesc_across(ot + ks * 16 * 128, N == 128 ? kTile : 0);
                mma_bf16_ss(leader, tm + L::kO, ad, sdesc_across(ph + ks * 16 * 128, kTile), id, ks < 3);
                mma_bf16_ss(leader, tm + L::kO, ad, sdesc_across(ph + kTile + ks * 16 * 128, kTile), id, 1);
            }
#pragma unroll
            for (int half = 0; half < L::kHalves; ++half) {  // x
                if (half == 0) ptx::named_sync<kPairs, kColsThreads>();
                else ptx::named_sync<kPairs + 1, kColsThreads>();
                if (half == 0 && i > 0) ptx::named_sync<kOutRead, L::kOut + 32>();  // dv has been read
                ptx::tc_fence_after_sync();
#pragma unroll
                for (int jj = 0; jj < 4; ++jj) {
                    const int j = half * 4 + jj;
                    const uint64_t bd = ptx::sdesc_sw128(kq + half * 2 * kTile + jj * 32);
                    mma_bf16(leader, tm + L::kX, tm + L::kPairS + 8 * j, bd, kAlong, j > 0);
                    mma_bf16(leader, tm + L::kX, tm + L::kPairS + N / 2 + 8 * j, bd, kAlong, 1);
                }
            }
            commit(leader, bar0 + 8 * kXDone);

            ptx::named_sync<kAdjoint, L::kWorkers + 32>();
            ptx::tc_fence_after_sync();
#pragma unroll
            for (int ks = 3; ks >= 0; --ks) {  // dv, in x's place
                const uint32_t id = idesc_bf16(128, 16 * (ks + 1), true);
                const uint64_t t0 = sdesc_across(th + ks * 16 * 128, kTile), t1 = sdesc_across(th + kTile + ks * 16 * 128, kTile);
                mma_bf16(leader, tm + L::kX, tm + L::kPairB + 8 * ks, t0, id, ks < 3);
                mma_bf16(leader, tm + L::kX, tm + L::kPairB + 32 + 8 * ks, t0, id, 1);
                mma_bf16(leader, tm + L::kX, tm + L::kPairB + 8 * ks, t1, id, 1);
                mma_bf16(leader, tm + L::kX, tm + L::kPairB + 32 + 8 * ks, t1, id, 1);
                mma_bf16(leader, tm + L::kX, tm + L::kPairB + 8 * ks, sdesc_across(th + 2 * kTile + ks * 16 * 128, kTile), id, 1);
            }
            commit(leader, bar0 + 8 * kDvDone);

            ptx::named_sync<kUpdate, L::kWorkers + 32>();
            ptx::tc_fence_after_sync();
#pragma unroll
            for (int half = 0; half < L::kHalves; ++half) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t kd = sdesc_across(kq + half * 2 * kTile + ks * 16 * 128, 2 * kTile);
                    const uint64_t qd = sdesc_across(kq + half * 2 * kTile + kTile + ks * 16 * 128, 2 * kTile);
                    mma_bf16(leader, tm + L::kS + half * 64, tm + L::kPairS + 8 * ks, qd, kAcross, 1);
                    mma_bf16(leader, tm + L::kS + half * 64, tm + L::kPairS + 32 + 8 * ks, qd, kAcross, 1);
                    mma_bf16(leader, tm + L::kS + half * 64, tm + L::kPairC + 8 * ks, kd, kAcross, 1);
                    mma_bf16(leader, tm + L::kS + half * 64, tm + L::kPairC + 32 + 8 * ks, kd, kAcross, 1);
                }
                commit(leader, bar0 + 8 * (kG0Done + half));
            }
            commit(leader, bar0 + 8 * (kDone0 + (i & 1)));
        }
        // nobody else waits for the last chunks': their arrivals must not find another CTA's memory
        for (int i = max(n_chunks - 2, 0); i < n_chunks; ++i) wait(kDone0 + (i & 1), i >> 1);
        ptx::named_sync<kLast, L::kWorkers + L::kOut + 32>();  // the last of it has been read
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tm, 512);
        return;
    }

    const int v = (warp & 3) * 32 + lane;  // this thread's row: a value column of the head
    const uint32_t tl = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16);

    if (warp >= L::kOutWarp) {
        const bool first = warp == L::kOutWarp && lane == 0;
#pragma unroll 1
        for (int i = 0; i < n_chunks; ++i) {
            const int c = n_chunks - 1 - i, t0 = bos + c * C;
            unsigned char *kept = keep.at((slot0 + c) * f.Hv + h, N);
            const bool whole = t0 + C <= eos;
            ptx::named_sync<kPairsOut, L::kWorkers + L::kOut>();  // G in pairs
            ptx::tc_fence_after_sync();
            keep_pairs<N, kOutOnly>(tl + L::kPairS, smem + St::kOutAt, kept + gdr_off_adjoint(N), kept + gdr_off_adjoint(N) + 2 * N * N,
                                    v, first);
            ptx::tc_fence_before_sync();
            ptx::named_arrive<kPairsRead, L::kWorkers + L::kOut>();
            if (first) ptx::bulk_wait_read<0>();  // the store before has read the staging rows
            ptx::named_sync<kOutOnly, L::kOut>();
            wait(kDvDone, i);
#pragma unroll 1
            for (int part = 0; part < C; part += 32) {
                float x[32];
                uint32_t hi[16], lo[16];
                tm_ld<32>(tl + L::kX + part, x);
                if (part == 32 && i + 1 < n_chunks) {
                    ptx::tc_fence_before_sync();
                    ptx::named_arrive<kOutRead, L::kOut + 32>();
                }
                split_row<32>(x, hi, lo);
                put_column<16>(smem + St::kOutAt + C * N * 2, v, part, lo);
                if (whole) {
                    __nv_bfloat16 *row = reinterpret_cast<__nv_bfloat16 *>(smem + St::kOutAt) + part * N + v;
#pragma unroll
                    for (int t = 0; t < 32; ++t) row[t * N] = __float2bfloat16_rn(x[t]);
                } else {
                    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(p.dv) + (static_cast<long long>(t0 + part) * f.Hv + h) * N + v;
#pragma unroll
                    for (int t = 0; t < 32; ++t)
                        if (t0 + part + t < eos) out[static_cast<long long>(t) * f.Hv * N] = __float2bfloat16_rn(x[t]);
                }
            }
            ptx::fence_proxy_async_smem();
            ptx::named_sync<kOutOnly, L::kOut>();
            if (first) {
                if (whole) ptx::tma_store_2d(&maps.o, h * N, t0, base + St::kOutAt);
                ptx::bulk_store(kept + gdr_off_dv(N), base + St::kOutAt + C * N * 2, C * N * 2);
                ptx::bulk_commit();
            }
        }
        if (first) ptx::bulk_wait<0>();
        ptx::tc_fence_before_sync();
        ptx::named_arrive<kLast, L::kWorkers + L::kOut + 32>();
        return;
    }
    if (!L::worker(warp)) return;

    const int wt = L::index(warp, lane), cg = warp >> 2;
    const int k0 = cg * L::kCols, tk0 = cg * L::kTok, half = k0 / 64;
    // G^T: row v, columns k
#pragma unroll 1
    for (int part = 0; part < L::kCols; part += L::kPart) {
        float x[L::kPart];
#pragma unroll
        for (int j = 0; j < L::kPart; ++j)
            x[j] = p.d_final_state ? p.d_final_state[s_at + static_cast<long long>(k0 + part + j) * N + v] : 0.f;
        tm_stf<L::kPart>(tl + L::kS + k0 + part, x);
    }
    ptx::tmem_wait_st();

#pragma unroll 1
    for (int i = 0; i < n_chunks; ++i) {
        const uint32_t stage = (i & 1) * St::kBytes;
        const float *vec = vec_of(i);
        const int c = n_chunks - 1 - i;
        wait_full(i);
        if (i == 0) {
            const int len = eos - (bos + c * C);
            if (len < C) {  // rows behind the sequence are another one's: zeros instead
                const uint4 z = make_uint4(0, 0, 0, 0);
                for (int e = len * (N / 8) + wt; e < C * (N / 8); e += L::kWorkers) {
                    const int row = e / (N / 8), col = (e % (N / 8)) * 8;
                    *reinterpret_cast<uint4 *>(smem + stage + St::kKQ + tile_off<2 * C>(row, col)) = z;
                    *reinterpret_cast<uint4 *>(smem + stage + St::kKQ + tile_off<2 * C>(C + row, col)) = z;
                    *reinterpret_cast<uint4 *>(smem + stage + St::kO + tile_off<C>(row, col)) = z;
                }
                ptx::fence_proxy_async_smem();
            }
            ptx::named_sync<kTail, L::kWorkers + 32>();
        }
        const float dc = vec[C - 1];
        if (i > 0) wait(kG0Done + half, i - 1);
        if (L::kHalves > 1 && half == 0 && i > 0) wait(kG1Done, i - 1);  // the update's left operands lie where pairs go
#pragma unroll
        for (int part = 0; part < L::kCols; part += L::kPart) {
            float x[L::kPart];
            uint32_t hi[L::kPart / 2], lo[L::kPart / 2];
            tm_ld<L::kPart>(tl + L::kS + k0 + part, x);
            split_row<L::kPart>(x, hi, lo);
            tm_st<L::kPart / 2>(tl + L::kPairS + (k0 + part) / 2, hi);
            tm_st<L::kPart / 2>(tl + L::kPairS + N / 2 + (k0 + part) / 2, lo);
#pragma unroll
            for (int j = 0; j < L::kPart; j += 2) mul2(x[j], x[j + 1], dc);
            tm_stf<L::kPart>(tl + L::kS + k0 + part, x);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before_sync();
        if (half == 0) ptx::named_arrive<kPairs, kColsThreads>();
        else ptx::named_arrive<kPairs + 1, kColsThreads>();
        ptx::named_arrive<kPairsOut, L::kWorkers + L::kOut>();

        float x[L::kTok];
        uint32_t hi[L::kTok / 2], lo[L::kTok / 2];
        wait(kXDone, i);
        {
            float y[L::kTok];
            tm_ld<L::kTok>(tl + L::kX + tk0, x);
            tm_ld<L::kTok>(tl + L::kO + tk0, y);
#pragma unroll
            for (int j = 0; j < L::kTok; j += 4) {
                const float4 e = *reinterpret_cast<const float4 *>(vec + C + tk0 + j);
                x[j] = fmaf(e.x, x[j], y[j]);
                x[j + 1] = fmaf(e.y, x[j + 1], y[j + 1]);
                x[j + 2] = fmaf(e.z, x[j + 2], y[j + 2]);
                x[j + 3] = fmaf(e.w, x[j + 3], y[j + 3]);
            }
        }
        split_row<L::kTok>(x, hi, lo);
        tm_st<L::kTok / 2>(tl + L::kPairB + tk0 / 2, hi);
        tm_st<L::kTok / 2>(tl + L::kPairB + 32 + tk0 / 2, lo);
        ptx::tmem_wait_st();
        ptx::tc_fence_before_sync();
        ptx::named_arrive<kAdjoint, L::kWorkers + 32>();

        // scale d dO, while dv is formed
        const unsigned char *orow = smem + stage + St::kO + (v >> 6) * kTile + (v & 7) * 2;
        const int chunk16 = (v >> 3) & 7;
#pragma unroll
        for (int j = 0; j < L::kTok; ++j) {
            const int t = tk0 + j;
            x[j] = __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(orow + t * 128 + ((chunk16 ^ (t & 7)) << 4)));
        }
#pragma unroll
        for (int j = 0; j < L::kTok; j += 4) {
            const float4 d = *reinterpret_cast<const float4 *>(vec + tk0 + j);
            x[j] *= d.x * f.scale; x[j + 1] *= d.y * f.scale; x[j + 2] *= d.z * f.scale; x[j + 3] *= d.w * f.scale;
        }
        split_row<L::kTok>(x, hi, lo);
        ptx::named_sync<kPairsRead, L::kWorkers + L::kOut>();
        ptx::tc_fence_after_sync();
        tm_st<L::kTok / 2>(tl + L::kPairS + tk0 / 2, hi);
        tm_st<L::kTok / 2>(tl + L::kPairS + 32 + tk0 / 2, lo);

        wait(kDvDone, i);
        tm_ld<L::kTok>(tl + L::kX + tk0, x);
#pragma unroll
        for (int j = 0; j < L::kTok; j += 4) {
            const float4 d = *reinterpret_cast<const float4 *>(vec + tk0 + j);
            x[j] *= -d.x; x[j + 1] *= -d.y; x[j + 2] *= -d.z; x[j + 3] *= -d.w;
        }
        split_row<L::kTok>(x, hi, lo);
        tm_st<L::kTok / 2>(tl + L::kPairC + tk0 / 2, hi);
        tm_st<L::kTok / 2>(tl + L::kPairC + 32 + tk0 / 2, lo);
        ptx::tmem_wait_st();
        ptx::tc_fence_before_sync();
        ptx::named_arrive<kUpdate, L::kWorkers + 32>();
    }
    wait(kG0Done + half, n_chunks - 1);
    if (p.d_initial_state) {
#pragma unroll 1
        for (int part = 0; part < L::kCols; part += L::kPart) {
            float x[L::kPart];
            tm_ld<L::kPart>(tl + L::kS + k0 + part, x);
#pragma unroll
            for (int j = 0; j < L::kPart; ++j) p.d_initial_state[s_at + static_cast<long long>(k0 + part + j) * N + v] = x[j];
        }
    }
    ptx::tc_fence_before_sync();
    ptx::named_arrive<kLast, L::kWorkers + L::kOut + 32>();
}

// Both chains of every (sequence, value head), which need nothing from one another: the reverse ones
// first, as they take longer.  One after the other, six documents to 300 tokens took 66 us a call
// instead of 45 (47 now); where HBM bounds them, the same.
template <int N>
__global__ void __launch_bounds__(Chain<N>::kWarps * 32)
gdr_backward_chains_kernel(const GdrBackwardArgs p, const __grid_constant__ GdrMaps maps, const unsigned char *__restrict__ prep,
                           const int32_t *__restrict__ order, const GdrChainStore keep) {
    if (blockIdx.y == 0) reverse_chain<N>(p, maps, prep, order, keep);
    else forward::chain<N, forward::kKeepMode>(p.f, maps, prep, order, keep, forward::Segments{1, false, nullptr});
}

// ------------------------------------------------------------------ the gradients of a chunk
//
// One CTA per (chunk, query/key head), the products on tcgen05 with 128 rows: row t of dq beside
// row t of dk.  With A = [dO; dv], the rows of Q beside those of K, per value head:
//
//   [X; M] = A err^T      [q k; k k] = [Q; K] K^T        then D and E elementwise, and their sums
//   [Y; H] = A S0^T       into dq, dk with the row's d, and q . Y, k . H
//   Z = [0; e' err] G^T   into dk with beta, and k . Z
//   [D; E] K + [0; D^T] Q + [0; E^T] K
//
// Sixteen warps hold dq and dk in registers over the heads that share them, four threads a row,
// and take each product out of tensor memory once (with eight, half of the issue slots stayed
// empty: 494 us where this took 437, and takes 443); one issues the MMAs and the copies, and one sums a
// head's dbeta and dg while the others go on to the next.  S0 and G (128 KB as pairs) do not fit
// beside the rest at once with the next head's: of two places one has S0, and the other err, dO
// and dv until those are in tensor memory, then G.  The next head has them the other way round,
// so that its err, dO and dv come once S0 has been used, while G still is.
// At 4 x 4096 tokens, 16 query/key and 32 value heads of 128, that is 12,000 clocks per chunk and
// head, of which the MMAs alone would take 5,800: they, the threads and the copies share the 128
// bytes a clock of shared memory (about 1 MB per chunk and head, two thirds of the time).
// Reading ahead into L2 changes nothing.
constexpr int kGradWarps = 16;  // and one for the MMAs and copies, one for the sums
constexpr int kGradThreads = kGradWarps * 32 + 64;

template <int N>
struct Grad {
    static constexpr uint32_t kRows = 0;                       // Q rows 0-63, K rows 64-127, [128][64] blocks
    static constexpr uint32_t kPlace = kRows + 2 * C * N * 2;  // two: S0 hi, lo [N][N]; and err hi, lo [64][N], dO, dv
    static constexpr uint32_t kPlaceBytes = 8 * C * N > 4 * N * N ? 8 * C * N : 4 * N * N;  // rows [128][N], then G hi, lo [N][N]
    static constexpr uint32_t kOv = 2 * C * N * 2;             // dO and dv behind err
    static constexpr uint32_t kZero = kPlace + 2 * kPlaceBytes;  // a tile of zeros
    static constexpr uint32_t kD = kZero + kTile;              // dv lo [64][N], then [D; E] hi, lo [128][64]
    static constexpr uint32_t kVec = kD + 4 * kTile;           // the prep's vectors, twice
    static constexpr uint32_t kBytes = kVec + 2 * 2048;
};

template <int N>
__global__ void __launch_bounds__(kGradThreads)
gdr_backward_grad_kernel(const GdrBackwardArgs p, const __grid_constant__ GdrMaps maps, const unsigned char *__restrict__ prep,
                         const GdrChainStore keep) {
    using M = Grad<N>;
    constexpr int kThreads = kGradWarps * 32, kGroups = kGradWarps / 4, kCols = N / kGroups;  // a thread's columns of its row
    constexpr uint32_t kT1 = 0, kT2 = 128, kT4 = 192, kA = 256, kB = 384;  // TMEM columns: Y/H or Z; X/M; gram; A; e' err
    enum { kRowsIn, kSpanIn, kStateIn, kAdjointIn, kX, kY, kD5, kZ, kGradBars };
    enum { kLeft = 1, kErrTaken, kTiles, kTaken, kInner, kSums };  // named barriers
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(8) unsigned long long bars[kGradBars];
    __shared__ uint32_t s_tmem;
    struct Sums {
        float row_a[kGroups][2 * C], row_z[kGroups][C], row_x[kGroups][2 * C], col_x[4][C], inner[kGradWarps];
    };
    __shared__ Sums both[2];  // of a head, and of the one after it
    const GdrPrefillArgs &f = p.f;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slot = blockIdx.x, hk = blockIdx.y, rep = f.Hv / f.Hk;
    const int b = gdr_find_seq(f.cu_seqlens, f.num_seqs, slot, lane);
    int bos, eos;
    if (!gdr_seq_bounds(f.cu_seqlens, f.num_seqs, f.T_total, b, bos, eos)) return;
    const int chunk = slot - ((bos >> 6) + b);
    if (chunk < 0 || chunk >= (eos - bos + C - 1) / C) return;
    const int t0 = bos + chunk * C, len = min(C, eos - t0);
    const long long item0 = static_cast<long long>(slot) * f.Hv + hk * rep;

    const uint32_t base = ptx::smem_addr(smem), bar0 = ptx::smem_addr(bars);
    if (warp == kGradWarps) {
        ptx::tmem_alloc(ptx::smem_addr(&s_tmem), 512);
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < kGradBars; ++i) ptx::mbar_init(bar0 + 8 * i, 1);
            ptx::fence_mbar_init();
        }
    }
    for (int i = tid; i < static_cast<int>(kTile) / 16; i += kGradThreads) reinterpret_cast<uint4 *>(smem + M::kZero)[i] = make_uint4(0, 0, 0, 0);
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    ptx::grid_dep_wait();
    const uint32_t tm = s_tmem;
    bool dead = false;  // a wait has run out: it is reported, and this thread waits no more
    auto wait = [&](int bar, int phase) {
        if (!dead && !wait_phase(bar0 + 8 * bar, phase & 1, kMaxPolls)) {
            dead = true;
            report(f.status, kDevTimeout);
        }
        ptx::tc_fence_after_sync();
    };

    if (warp == kGradWarps) {
        const uint32_t leader = elect_lane();
        auto load_span = [&](int r) {
            if (lane == 0) {
                const unsigned char *src = keep.at(item0 + r, N);
                const uint32_t span = bar0 + 8 * kSpanIn, at = base + M::kPlace + (r & 1) * M::kPlaceBytes;
                const int h = hk * rep + r;
                ptx::mbar_arrive_expect_tx(span, 5 * C * N * 2 + kVecKept * 4);
                ptx::bulk_load(at, src + gdr_off_err(N), 2 * C * N * 2, span);
#pragma unroll
                for (int j = 0; j < N / 64; ++j) {
                    ptx::tma_load_2d(at + M::kOv + j * 2 * kTile, &maps.d_o, h * N + j * 64, t0, span);
                    ptx::tma_load_2d(at + M::kOv + j * 2 * kTile + kTile, &maps.dv, h * N + j * 64, t0, span);
                }
                ptx::bulk_load(base + M::kD, src + gdr_off_dv(N), C * N * 2, span);
                ptx::bulk_load(base + M::kVec + (r & 1) * 2048, prep + (item0 + r) * kGdrPrepBytes + kGdrPrepVec, kVecKept * 4, span);
            }
            __syncwarp();
        };
        auto load_square = [&](int bar, uint32_t at, const unsigned char *src) {  // S0 or G
            if (lane == 0) {
                ptx::mbar_arrive_expect_tx(bar0 + 8 * bar, 4 * N * N);
                ptx::bulk_load(at, src, 4 * N * N, bar0 + 8 * bar);
            }
            __syncwarp();
        };
        if (lane == 0) {
            ptx::mbar_arrive_expect_tx(bar0 + 8 * kRowsIn, 2 * C * N * 2);
#pragma unroll
            for (int j = 0; j < N / 64; ++j) {
                ptx::tma_load_2d(base + M::kRows + j * 2 * kTile, &maps.q, hk * N + j * 64, t0, bar0 + 8 * kRowsIn);
                ptx::tma_load_2d(base + M::kRows + j * 2 * kTile + kTile, &maps.k, hk * N + j * 64, t0, bar0 + 8 * kRowsIn);
            }
        }
        __syncwarp();
        load_span(0);
        load_square(kStateIn, base + M::kPlace + M::kPlaceBytes, keep.at(item0, N) + gdr_off_state());
        constexpr uint32_t kAlong64 = idesc_bf16(128, 64, false), kAcrossN = idesc_bf16(128, N, true);
        constexpr uint32_t kLeftAcross = 1u << 15;
        const uint32_t rows = base + M::kRows, krows = rows + kTile;
        const uint32_t dt = base + M::kD, zt = base + M::kZero;
#pragma unroll 1
        for (int r = 0; r < rep; ++r) {
            const uint32_t et = base + M::kPlace + (r & 1) * M::kPlaceBytes, gt = et, st = base + M::kPlace + (~r & 1) * M::kPlaceBytes;
            ptx::named_sync<kLeft, kThreads + 32>();  // A in tensor memory
            ptx::tc_fence_after_sync();
#pragma unroll
            for (int j = 0; j < N / 16; ++j)  // [q k; k k]
                mma_bf16_ss(leader, tm + kT4, ptx::sdesc_sw128(rows + (j >> 2) * 2 * kTile + (j & 3) * 32),
                            ptx::sdesc_sw128(krows + (j >> 2) * 2 * kTile + (j & 3) * 32), kAlong64, j > 0);
#pragma unroll
            for (int j = 0; j < N / 16; ++j) {  // [X; M]
                const uint64_t hd = ptx::sdesc_sw128(et + (j >> 2) * kTile + (j & 3) * 32);
                const uint64_t ld = ptx::sdesc_sw128(et + C * N * 2 + (j >> 2) * kTile + (j & 3) * 32);
                mma_bf16(leader, tm + kT2, tm + kA + 8 * j, hd, kAlong64, j > 0);
                mma_bf16(leader, tm + kT2, tm + kA + N / 2 + 8 * j, hd, kAlong64, 1);
                mma_bf16(leader, tm + kT2, tm + kA + 8 * j, ld, kAlong64, 1);
            }
            commit(leader, bar0 + 8 * kX);
            wait(kStateIn, r);
#pragma unroll
            for (int j = 0; j < N / 16; ++j) {  // [Y; H]
                const uint64_t hd = sdesc_across(st + j * 16 * 128, N * 128), ld = sdesc_across(st + 2 * N * N + j * 16 * 128, N * 128);
                mma_bf16(leader, tm + kT1, tm + kA + 8 * j, hd, kAcrossN, j > 0);
                mma_bf16(leader, tm + kT1, tm + kA + N / 2 + 8 * j, hd, kAcrossN, 1);
                mma_bf16(leader, tm + kT1, tm + kA + 8 * j, ld, kAcrossN, 1);
            }
            commit(leader, bar0 + 8 * kY);
            wait(kX, r);  // err has been read by the MMAs, dO and dv before that by the threads,
            ptx::named_sync<kErrTaken, kThreads + 32>();  // and err too: e' err is in tensor memory
            load_square(kAdjointIn, gt, keep.at(item0 + r, N) + gdr_off_adjoint(N));
            ptx::named_sync<kTiles, kThreads + 32>();  // D and E written, X, M and the gram read
            ptx::tc_fence_after_sync();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                const uint64_t kd = sdesc_across(krows + ks * 16 * 128, 2 * kTile), qd = sdesc_across(rows + ks * 16 * 128, 2 * kTile);
#pragma unroll
                for (int part = 0; part < 2; ++part) {  // high, low
                    const uint32_t d = dt + part * 2 * kTile;
                    mma_bf16_ss(leader, tm + kT2, ptx::sdesc_sw128(d + ks * 32), kd, kAcrossN, ks + part > 0);
                    // rows 64 - 127 the tile's columns, rows 0 - 63 the zeros that lie before it
                    const uint32_t zero = zt + ks * 16 * 128, to_d = d - zt, to_e = to_d + kTile;
                    mma_bf16_ss(leader, tm + kT2, sdesc_across(zero, to_d), qd, kAcrossN | kLeftAcross, 1);
                    mma_bf16_ss(leader, tm + kT2, sdesc_across(zero, to_e), kd, kAcrossN | kLeftAcross, 1);
                }
            }
            commit(leader, bar0 + 8 * kD5);
            ptx::named_sync<kTaken, kThreads + 32>();  // Y and H read
            wait(kAdjointIn, r);
#pragma unroll
            for (int j = 0; j < N / 16; ++j) {  // Z
                const uint64_t hd = sdesc_across(gt + j * 16 * 128, N * 128), ld = sdesc_across(gt + 2 * N * N + j * 16 * 128, N * 128);
                mma_bf16(leader, tm + kT1, tm + kB + 8 * j, hd, kAcrossN, j > 0);
                mma_bf16(leader, tm + kT1, tm + kB + N / 2 + 8 * j, hd, kAcrossN, 1);
                mma_bf16(leader, tm + kT1, tm + kB + 8 * j, ld, kAcrossN, 1);
            }
            commit(leader, bar0 + 8 * kZ);
            ptx::named_sync<kInner, kThreads + 64>();  // S0 and G read by the threads, the vectors of the head before by the sums
            if (r + 1 < rep) {
                wait(kD5, r);  // D and E, and S0 before them, have been read by the MMAs
                load_span(r + 1);
                wait(kZ, r);  // and G
                load_square(kStateIn, gt, keep.at(item0 + r + 1, N) + gdr_off_state());
            }
        }
        __syncthreads();
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tm, 512);
        return;
    }

    if (warp == kGradWarps + 1) {  // dbeta, dgam and its sums from the end: tokens 2 lane, 2 lane + 1
#pragma unroll 1
        for (int r = 0; r < rep; ++r) {
            const Sums &sums = both[r & 1];
            const float *vec = reinterpret_cast<const float *>(smem + M::kVec + (r & 1) * 2048);
            wait(kSpanIn, r);
            ptx::named_arrive<kInner, kThreads + 64>();
            ptx::named_sync<kSums, kThreads + 32>();
            float db[2], dgam[2], ys = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int u = 2 * lane + j;
                float kz = 0.f, rows = 0.f;  // e' k . Z
#pragma unroll
                for (int c = 0; c < kGroups; ++c) {
                    kz += sums.row_z[c][u];
                    rows += (sums.row_x[c][u] + sums.row_x[c][C + u]) + (sums.row_a[c][u] + sums.row_a[c][C + u]);
                }
                db[j] = (sums.col_x[0][u] + sums.col_x[1][u]) + (sums.col_x[2][u] + sums.col_x[3][u]) + kz;
                dgam[j] = rows - vec[kVecBeta + u] * db[j];
                ys = fmaf(vec[kVecBeta + u], kz, ys);
            }
#pragma unroll
            for (int off = 16; off; off >>= 1) ys += __shfl_xor_sync(0xffffffffu, ys, off);
            if (lane == 31) {
                float gs = 0.f;
#pragma unroll
                for (int w = 0; w < kGradWarps; ++w) gs += sums.inner[w];
                dgam[1] += ys + vec[kVecD + C - 1] * gs;
            }
            float sum = dgam[0] + dgam[1];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float o = __shfl_down_sync(0xffffffffu, sum, off);
                if (lane + off < 32) sum += o;
            }
            const float out[2] = {sum, sum - dgam[0]};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int u = 2 * lane + j;
                if (u < len) {
                    const long long at = static_cast<long long>(t0 + u) * f.Hv + hk * rep + r;
                    p.dg[at] = out[j];
                    p.dbeta[at] = db[j];
                }
            }
        }
        __syncthreads();
        return;
    }

    const int row = (warp & 3) * 32 + lane, t = row & 63, cg = warp >> 2, c0 = cg * kCols;
    const bool lower = row >= C;  // a row of dk (dv, K) instead of dq (dO, Q)
    const uint32_t tl = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const unsigned char *own = smem + M::kRows;  // this thread's row of Q or K
    float acc[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
    wait(kRowsIn, 0);
    if (t >= len)  // a row behind the sequence is another one's: zeros instead
#pragma unroll
        for (int c = 0; c < kCols; c += 8) *reinterpret_cast<uint4 *>(smem + M::kRows + tile_off<2 * C>(row, c0 + c)) = make_uint4(0, 0, 0, 0);

    // sum of x[i] times this thread's row of Q or K, columns col ..
    auto dot_row = [&](const float (&x)[16], int col) {
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < 16; c += 8) {
            const uint4 u = *reinterpret_cast<const uint4 *>(own + tile_off<2 * C>(row, col + c));
            s = fmaf(low(u.x), x[c], s); s = fmaf(high(u.x), x[c + 1], s);
            s = fmaf(low(u.y), x[c + 2], s); s = fmaf(high(u.y), x[c + 3], s);
            s = fmaf(low(u.z), x[c + 4], s); s = fmaf(high(u.z), x[c + 5], s);
            s = fmaf(low(u.w), x[c + 6], s); s = fmaf(high(u.w), x[c + 7], s);
        }
        return s;
    };

#pragma unroll 1
    for (int r = 0; r < rep; ++r) {
        const float *vec = reinterpret_cast<const float *>(smem + M::kVec + (r & 1) * 2048);
        const unsigned char *span = smem + M::kPlace + (r & 1) * M::kPlaceBytes, *state = smem + M::kPlace + (~r & 1) * M::kPlaceBytes;
        Sums &sums = both[r & 1];
        wait(kSpanIn, r);
        // A's row: dO as it is, or dv's pair; and beside the products with it e' err
        {
            uint32_t hi[kCols / 2], lo[kCols / 2];
#pragma unroll
            for (int i = 0; i < kCols / 8; ++i) {
                uint4 x = make_uint4(0, 0, 0, 0), y = x;
                if (t < len) x = *reinterpret_cast<const uint4 *>(span + M::kOv + tile_off<2 * C>(row, c0 + 8 * i));
                if (lower && t < len) y = *reinterpret_cast<const uint4 *>(smem + M::kD + tile_off<C>(t, c0 + 8 * i));
                hi[4 * i] = x.x; hi[4 * i + 1] = x.y; hi[4 * i + 2] = x.z; hi[4 * i + 3] = x.w;
                lo[4 * i] = y.x; lo[4 * i + 1] = y.y; lo[4 * i + 2] = y.z; lo[4 * i + 3] = y.w;
            }
            tm_st<kCols / 2>(tl + kA + c0 / 2, hi);
            tm_st<kCols / 2>(tl + kA + N / 2 + c0 / 2, lo);
            ptx::tmem_wait_st();
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_before_sync();
            ptx::named_arrive<kLeft, kThreads + 32>();
            const float e = vec[kVecE1 + t];
#pragma unroll
            for (int i = 0; i < kCols / 8; ++i) {
                uint4 x = make_uint4(0, 0, 0, 0), y = x;
                if (lower) {
                    x = *reinterpret_cast<const uint4 *>(span + tile_off<C>(t, c0 + 8 * i));
                    y = *reinterpret_cast<const uint4 *>(span + C * N * 2 + tile_off<C>(t, c0 + 8 * i));
                }
                split(e * (low(x.x) + low(y.x)), e * (high(x.x) + high(y.x)), hi[4 * i], lo[4 * i]);
                split(e * (low(x.y) + low(y.y)), e * (high(x.y) + high(y.y)), hi[4 * i + 1], lo[4 * i + 1]);
                split(e * (low(x.z) + low(y.z)), e * (high(x.z) + high(y.z)), hi[4 * i + 2], lo[4 * i + 2]);
                split(e * (low(x.w) + low(y.w)), e * (high(x.w) + high(y.w)), hi[4 * i + 3], lo[4 * i + 3]);
            }
            tm_st<kCols / 2>(tl + kB + c0 / 2, hi);
            tm_st<kCols / 2>(tl + kB + N / 2 + c0 / 2, lo);
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            ptx::named_arrive<kErrTaken, kThreads + 32>();
        }

        // D (row t, columns s <= t) from X and q k, or E (s < t) from M and k k, and their sums
        wait(kX, r);
        {
            constexpr int kTok = C / kGroups;  // columns: tokens
            const int s0 = cg * kTok;
            const float ti = vec[kVecInt + t], tf = vec[kVecFrac + t], sign = lower ? -1.f : f.scale;
            const int last = lower ? t - 1 : t;
            float z[kTok], x[kTok], gram[kTok], rows_sum = 0.f;
            tm_ld<kTok>(tl + kT2 + s0, x);
            tm_ld<kTok>(tl + kT4 + s0, gram);
#pragma unroll
            for (int q = 0; q < kTok; q += 4) {
                const float4 si = *reinterpret_cast<const float4 *>(vec + kVecInt + s0 + q), sf = *reinterpret_cast<const float4 *>(vec + kVecFrac + s0 + q);
                const float4 sb = *reinterpret_cast<const float4 *>(vec + kVecBeta + s0 + q);
                const float whole[4] = {si.x, si.y, si.z, si.w}, part[4] = {sf.x, sf.y, sf.z, sf.w}, beta[4] = {sb.x, sb.y, sb.z, sb.w};
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int i = q + m;
                    const float w = exp2_flush((ti - whole[m]) + (tf - part[m]));
                    const float wx = gdr::keep(s0 + i <= last, sign * w * x[i]);
                    z[i] = gdr::keep(s0 + i <= last, wx * gram[i]);
                    x[i] = beta[m] * wx;
                    rows_sum = fmaf(beta[m], z[i], rows_sum);
                }
            }
            uint32_t hi[kTok / 2], lo[kTok / 2];
            split_row<kTok>(x, hi, lo);
            store_row<2 * C>(smem + M::kD, smem + M::kD + 2 * kTile, row, s0, hi, lo);
            sums.row_x[cg][row] = rows_sum;
            // column sums over the warp's rows: each step adds and halves the columns a lane carries
#pragma unroll
            for (int m = kTok / 2; m >= 1; m >>= 1) {
                const bool up = lane & m;
#pragma unroll
                for (int i = 0; i < m; ++i) {
                    const float send = up ? z[i] : z[i + m], mine = up ? z[i + m] : z[i];
                    z[i] = mine + __shfl_xor_sync(0xffffffffu, send, m);
                }
            }
            static_assert(kTok == 16, "two lanes are left with each column");
            z[0] += __shfl_xor_sync(0xffffffffu, z[0], 16);
            if (lane < kTok) sums.col_x[warp & 3][s0 + lane] = z[0];
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before_sync();
        ptx::named_arrive<kTiles, kThreads + 32>();

        // Y or H
        wait(kY, r);
        {
            const float scale = lower ? -vec[kVecD + t] : f.scale * vec[kVecD + t];
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < kCols; c += 16) {
                float x[16];
                tm_ld<16>(tl + kT1 + c0 + c, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    x[i] *= scale;
                    acc[c + i] += x[i];
                }
                s += dot_row(x, c0 + c);
            }
            sums.row_a[cg][row] = s;
        }
        ptx::tc_fence_before_sync();
        ptx::named_arrive<kTaken, kThreads + 32>();

        // <G, S0>
        wait(kStateIn, r);
        wait(kAdjointIn, r);
        {
            float2 sum2 = make_float2(0.f, 0.f);
            const uint4 *gp = reinterpret_cast<const uint4 *>(span), *sp = reinterpret_cast<const uint4 *>(state);
            constexpr int kLow = 2 * N * N / 16;
#pragma unroll 2
            for (int i = tid; i < kLow; i += kThreads) {
                const uint4 a = gp[i], al = gp[i + kLow], y = sp[i], yl = sp[i + kLow];
                sum2 = fma2(add2(pair(a.x), pair(al.x)), add2(pair(y.x), pair(yl.x)), sum2);
                sum2 = fma2(add2(pair(a.y), pair(al.y)), add2(pair(y.y), pair(yl.y)), sum2);
                sum2 = fma2(add2(pair(a.z), pair(al.z)), add2(pair(y.z), pair(yl.z)), sum2);
                sum2 = fma2(add2(pair(a.w), pair(al.w)), add2(pair(y.w), pair(yl.w)), sum2);
            }
            float sum = sum2.x + sum2.y;
#pragma unroll
            for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            if (lane == 0) sums.inner[warp] = sum;
        }
        ptx::named_arrive<kInner, kThreads + 64>();

        wait(kD5, r);
#pragma unroll
        for (int c = 0; c < kCols; c += 16) {
            float x[16];
            tm_ld<16>(tl + kT2 + c0 + c, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[c + i] += x[i];
        }
        wait(kZ, r);
        if (lower) {
            const float beta = vec[kVecBeta + t];
            float s = 0.f;
#pragma unroll
            for (int c = 0; c < kCols; c += 16) {
                float x[16];
                tm_ld<16>(tl + kT1 + c0 + c, x);
                s += dot_row(x, c0 + c);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[c + i] = fmaf(beta, x[i], acc[c + i]);
            }
            sums.row_z[cg][t] = s;
        }
        ptx::tc_fence_before_sync();
        ptx::named_sync<kSums, kThreads + 32>();

    }

    if (t < len) {
        __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(lower ? p.dk : p.dq) + (static_cast<long long>(t0 + t) * f.Hk + hk) * N + c0;
#pragma unroll
        for (int c = 0; c < kCols; c += 8)
            *reinterpret_cast<uint4 *>(out + c) = make_uint4(pack(acc[c], acc[c + 1]), pack(acc[c + 2], acc[c + 3]),
                                                             pack(acc[c + 4], acc[c + 5]), pack(acc[c + 6], acc[c + 7]));
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
}

template <int N>
cudaError_t chains(const GdrBackwardArgs &p, const GdrMaps &maps, const unsigned char *prep, const int32_t *order,
                  GdrChainStore keep, cudaStream_t stream) {
    static std::atomic<unsigned long long> allowed{0};
    constexpr int kSmem = static_cast<int>(Stage<N>::kSmem > forward::Stage<N>::kSmem ? Stage<N>::kSmem : forward::Stage<N>::kSmem);
    static_assert(kSmem <= 226 * 1024, "two stages and the output rows fit one SM");
    const cudaError_t e = gdr_allow_smem(reinterpret_cast<const void *>(gdr_backward_chains_kernel<N>), kSmem, allowed);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(p.f.num_seqs) * static_cast<unsigned>(p.f.Hv), 2);
    return gdr_launch(gdr_backward_chains_kernel<N>, grid, Chain<N>::kWarps * 32, kSmem, stream, p.f.T_total > 0, p, maps, prep, order, keep);
}

template <int N>
cudaError_t grads(const GdrBackwardArgs &p, const GdrMaps &maps, const unsigned char *prep, GdrChainStore keep, cudaStream_t stream) {
    static std::atomic<unsigned long long> allowed{0};
    constexpr int kSmem = Grad<N>::kBytes;
    static_assert(kSmem <= 210 * 1024, "the tiles and the static sums fit one SM");
    const cudaError_t e = gdr_allow_smem(reinterpret_cast<const void *>(gdr_backward_grad_kernel<N>), kSmem, allowed);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(gdr_max_slots(p.f.num_seqs, p.f.T_total)), p.f.Hk);
    return gdr_launch(gdr_backward_grad_kernel<N>, grid, kGradThreads, kSmem, stream, true, p, maps, prep, keep);
}

}  // namespace

size_t gdr_backward_workspace_bytes(int num_seqs, int T_total, int Hv, int N) {
    return gdr_order_bytes(num_seqs) + 112 + gdr_prep_bytes(num_seqs, T_total, Hv) +
           static_cast<size_t>(gdr_max_slots(num_seqs, T_total)) * Hv * gdr_chain_bytes(N);
}

cudaError_t launch_gdr_prefill_backward(const GdrBackwardArgs &p, void *workspace, cudaStream_t s) {
    const GdrPrefillArgs &f = p.f;
    unsigned char *prep = gdr_behind_order(workspace, f.num_seqs);
    const GdrChainStore keep{prep + gdr_prep_bytes(f.num_seqs, f.T_total, f.Hv)};
    GdrMaps maps = {};
    if (!gdr_forward_maps(&maps, f)) return cudaErrorInvalidValue;
    if (f.T_total > 0 && !(make_tile_map(&maps.d_o, p.d_o, f.T_total, f.Hv, f.N) && make_tile_map(&maps.dv, p.dv, f.T_total, f.Hv, f.N) &&
                           make_plain_map(&maps.o, p.dv, true, f.T_total, f.Hv, f.N)))
        return cudaErrorInvalidValue;
    int32_t *order;
    cudaError_t e = launch_gdr_order(f, workspace, &order, s);
    if (e == cudaSuccess && f.T_total > 0) e = launch_gdr_prep(f, maps, prep, s);
    if (e != cudaSuccess) return e;
    e = f.N == 64 ? chains<64>(p, maps, prep, order, keep, s) : chains<128>(p, maps, prep, order, keep, s);
    if (e != cudaSuccess || f.T_total == 0) return e;
    return f.N == 64 ? grads<64>(p, maps, prep, keep, s) : grads<128>(p, maps, prep, keep, s);
}

}  // namespace wkv7
