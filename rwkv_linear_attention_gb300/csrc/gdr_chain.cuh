// The gated delta rule's chain over a sequence's chunks (bf16 inputs).  Per chunk, with That, P, d, e from gdr_prep.cuh:
//
//   err = That (V - d K S0)     o = scale d Q S0 + P err     S_C = d_C S0 + K^T (e err)
//
// One CTA per (sequence, value head), everything transposed: the rows of the MMAs are the N
// value columns v, so S^T (N x N, fp32) stays in tensor memory for the whole sequence and
// every left operand (S^T, r^T = (V - d K S0)^T, err^T, (e err)^T) is written to tensor
// memory by the thread that owns its row, while K, Q, That and P are right operands just as
// they lie in shared memory (K along its rows for K S0, across them for K^T err).
//
// Warps: eight workers on the chain, one that issues the MMAs, one that issues the copies
// (TMA, one chunk ahead), one per 32 rows for the outputs.  They hand over by named barriers
// (threads to MMAs) and mbarriers (commits and copies to threads).  Per chunk, the chain on
// the left, what runs beside it on the right:
//
//   S as pairs (first half of its          the second half of the update before it;
//     columns, then the second)            that chunk's o += P err, then o out
//   x = K S0, half by half                 S = d_C S, V into registers
//   r = V - d x as pairs
//   err = That r
//   e err as pairs                         o = Q S0, times scale d
//   S += K^T (e err)                       err as pairs
//
// Precision: K, Q and V are exact bf16; S, r, err and P are pairs of bf16, That has three terms
// (gdr_mma.cuh; gdr_prep.cuh says why), so each product is off by 2^-16 of its operands; sums are
// fp32 and S itself is never rounded.  One MMA per product instead of two or three would leave
// 2^-8 in the carried state.
#pragma once

#include "gdr_internal.cuh"
#include "gdr_tc.cuh"

namespace wkv7 {
namespace gdr {
namespace forward {

constexpr uint32_t kMaxPolls = 1u << 17;  // of up to 20 us: seconds

__device__ __forceinline__ float ld_state(const void *p, wkv7_dtype dt, long long i) {
    if (dt == WKV7_F32) return static_cast<const float *>(p)[i];
    if (dt == WKV7_BF16) return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
    return __half2float(static_cast<const __half *>(p)[i]);
}
__device__ __forceinline__ void st_state(void *p, wkv7_dtype dt, long long i, float x) {
    if (dt == WKV7_F32) static_cast<float *>(p)[i] = x;
    else if (dt == WKV7_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
    else static_cast<__half *>(p)[i] = __float2half_rn(x);
}

template <int N>
struct Stage {
    static constexpr uint32_t kKQ = 0;                  // K rows 0-63, Q rows 64-127, [128][64] blocks
    static constexpr uint32_t kV = 2 * C * N * 2;       // plain [64][N]
    static constexpr uint32_t kPrep = kV + C * N * 2;   // P, That, d, e
    static constexpr uint32_t kPrepBytes = kGdrPrepVec + 2 * C * 4;
    static constexpr uint32_t kBytes = kPrep + kGdrPrepVec + 1024;
    static constexpr uint32_t kOutAt = 2 * kBytes;      // o of one chunk, plain [64][N], fp32 or bf16
    static constexpr uint32_t kSmem = kOutAt + C * N * 4;
};

// mbarriers.  A wait for a phase must come before the phase after it ends; where a reader's own
// progress does not see to that, a barrier belongs to a stage (kFull, kDone: its next phase needs
// the stage filled again, which the reader's wait holds up).
enum Bar { kFull0, kFull1, kDone0, kDone1, kXDone, kErrDone, kODone, kS0Done, kS1Done, kBars };
// Named barriers: kPairs, + 1 (a half of S in pairs), then as they are used.
enum Named { kPairs = 1, kResidual = 3, kUpdate, kOutputs, kTail, kOutRead, kLast, kOutOnly };

// What a chain is run for: the call's outputs; the backward's first pass, which computes no outputs
// and keeps, per chunk, the state before it and err (pairs of bf16) for the gradients; or the last
// state alone.
enum Mode { kOutputsMode, kKeepMode, kStateMode };

// A sequence in segments of equal length (but see `half`) that run at once, for calls with few chains.  The state is
// carried linearly, S_end = A S_in + S_part, so a first pass runs segments 0 .. count - 2 for their
// last states alone: the first from the call's state, each other one from zero (S_part) and, without
// V, from the identity (A).  A small kernel chains the states that the segments start from, and the
// second pass runs all segments with outputs.  Slots of N x N floats per (sequence, head):
//   start of segments 0 .. count - 1, then S_part and A of segments 1 .. count - 2
// (segment 0's is a copy: the call's final state may be written over its initial one before
// that segment has read it)
struct Segments {
    int count;       // 1: whole sequences
    bool half;       // segment count - 2 has half the length of the others
    float *scratch;
    // the chunks of segment s of a sequence of `all` chunks
    __device__ void range(int all, int s, int &first, int &n) const {
        const int halves = half ? 2 * count - 1 : count, step = half ? 2 : 1, unit = (all + halves - 1) / halves;
        first = min((step * s - (half && s == count - 1 ? 1 : 0)) * unit, all);
        n = min((half && s == count - 2 ? 1 : step) * unit, all - first);
    }
    __host__ __device__ int slots() const { return 3 * count - 4; }
    __device__ float *slot(long long pair, int i, int n2) const { return scratch + (pair * slots() + i) * n2; }
    __device__ float *start(long long pair, int seg, int n2) const { return slot(pair, seg, n2); }
    __device__ float *part(long long pair, int seg, int n2) const { return slot(pair, count + (seg - 1), n2); }
    __device__ float *transfer(long long pair, int seg, int n2) const { return slot(pair, 2 * count - 2 + (seg - 1), n2); }
    __host__ __device__ int first_pass_runs() const { return 2 * count - 3; }
};

// One CTA's chain (`maps` lies in a kernel's parameters).
template <int N, Mode kMode>
__device__ __forceinline__ void chain(const GdrPrefillArgs &p, const GdrMaps &maps, const unsigned char *__restrict__ prep,
                                      const int32_t *__restrict__ order, const GdrChainStore &keep, const Segments &seg) {
    constexpr bool kStates = kMode != kOutputsMode, kKeep = kMode == kKeepMode;
    constexpr int kOuts = kMode == kStateMode ? 0 : Chain<N>::kOut;
    using L = Chain<N>;
    using St = Stage<N>;
    constexpr int kHalfThreads = L::kWorkers / L::kHalves + 32;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(8) unsigned long long bars[kBars];
    __shared__ uint32_t s_tmem;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x % p.Hv, rank = blockIdx.x / p.Hv, b = order ? order[rank] : gdr_by_length(p.cu_seqlens, p.num_seqs, rank, lane);
    int bos, eos;
    if (b < 0 || b >= p.num_seqs || !gdr_seq_bounds(p.cu_seqlens, p.num_seqs, p.T_total, b, bos, eos)) {
        if (threadIdx.x == 0 && h == 0) report(p.status, kDevBadSeqlens);
        return;
    }
    const long long pair = static_cast<long long>(b) * p.Hv + h;
    // this run's chunks, and where its state comes from and goes to
    const int all_chunks = (eos - bos + C - 1) / C;
    int chunk0 = 0, n_chunks = all_chunks;
    const void *from = p.initial_state;
    void *to = p.final_state;
    long long from_at = pair * (N * N), to_at = from_at;
    wkv7_dtype from_type = p.state_dtype, to_type = p.state_dtype;
    bool identity = false;
    if (seg.count > 1) {
        const int run = blockIdx.y;
        const int s = kMode == kStateMode ? (run + 1) >> 1 : run;
        seg.range(all_chunks, s, chunk0, n_chunks);
        if (kMode == kStateMode) {
            identity = run > 0 && (run & 1) == 0;
            if (run > 0) from = nullptr;
            to = run == 0 ? seg.start(pair, 1, N * N) : identity ? seg.transfer(pair, s, N * N) : seg.part(pair, s, N * N);
            to_at = 0;
            to_type = WKV7_F32;
        } else {
            if (s > 0 || from) {
                from = seg.start(pair, s, N * N);
                from_at = 0;
                from_type = WKV7_F32;
            }
            if (s + 1 < seg.count) to = nullptr;
        }
    }
    // element (k, v) of the state that the run starts from
    auto start = [&](int k, int v) {
        if (kMode == kStateMode && identity) return k == v ? 1.f : 0.f;
        return from ? ld_state(from, from_type, from_at + k * N + v) : 0.f;
    };
    if (n_chunks <= 0) {  // the state as it was
        ptx::grid_dep_wait();
        if (to)
            for (int i = threadIdx.x; i < N * N; i += L::kWarps * 32) st_state(to, to_type, to_at + i, start(i / N, i % N));
        return;
    }
    const int first_slot = bos >> 6;
    bos += chunk0 * C;
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
    const uint32_t tm = s_tmem;
    const int hk = h / (p.Hv / p.Hk);
    const long long slot0 = first_slot + b + chunk0;

    bool dead = false;  // a wait has run out: it is reported, and this thread waits no more
    auto wait = [&](int bar, int phase) {
        if (!dead && !wait_phase(bar0 + 8 * bar, phase & 1, kMaxPolls)) {
            dead = true;
            report(p.status, kDevTimeout);
        }
        ptx::tc_fence_after_sync();
    };
    // chunk c's last MMAs, and so all that they waited for
    auto wait_done = [&](int c) { wait(kDone0 + (c & 1), c >> 1); };
    auto vec_of = [&](int c) { return reinterpret_cast<const float *>(smem + (c & 1) * St::kBytes + St::kPrep + kGdrPrepVec); };

    if (warp == L::kLoadWarp) {
        if (lane == 0) {
#pragma unroll 1
            for (int c = 0; c < n_chunks; ++c) {
                if (c >= 2) wait_done(c - 2);  // the stage's chunk is through
                const uint32_t s = base + (c & 1) * St::kBytes, full = bar0 + 8 * (kFull0 + (c & 1));
                const int t0 = bos + c * C;
                constexpr uint32_t kSkip = kStates ? kGdrPrepThat : 0;  // P is for outputs alone
                ptx::mbar_arrive_expect_tx(full, (kStates ? 2 : 3) * C * N * 2 + St::kPrepBytes - kSkip);
#pragma unroll
                for (int j = 0; j < N / 64; ++j) {
                    ptx::tma_load_2d(s + St::kKQ + j * 2 * kTile, &maps.k, hk * N + j * 64, t0, full);
                    if (!kStates) ptx::tma_load_2d(s + St::kKQ + j * 2 * kTile + kTile, &maps.q, hk * N + j * 64, t0, full);
                }
                ptx::tma_load_2d(s + St::kV, &maps.v, h * N, t0, full);
                ptx::bulk_load(s + St::kPrep + kSkip, prep + ((slot0 + c) * p.Hv + h) * kGdrPrepBytes + kSkip, St::kPrepBytes - kSkip, full);
            }
        }
        return;
    }

    if (warp == L::kMmaWarp) {
        const uint32_t leader = elect_lane();
        constexpr uint32_t kRows = idesc_bf16(128, 64, false), kAcross = idesc_bf16(128, 64, true);
#pragma unroll 1
        for (int c = 0; c < n_chunks; ++c) {
            const uint32_t s = base + (c & 1) * St::kBytes;
            const uint32_t kq = s + St::kKQ, ph = s + St::kPrep, th = ph + kGdrPrepThat;
            // d (+)= pair B times a lower triangular tile of two or three terms
            auto lower = [&](uint32_t d, uint32_t tile, int terms, uint32_t first) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {  // tokens 16 ks .. reach columns 16 ks ..
                    const uint32_t id = idesc_bf16(128, 64 - 16 * ks, false);
                    const uint32_t row = tile + ks * 16 * 128 + ks * 32;
                    mma_bf16(leader, d + 16 * ks, tm + L::kPairB + 8 * ks, ptx::sdesc_sw128(row), id, ks > 0 ? 1u : first);
                    mma_bf16(leader, d + 16 * ks, tm + L::kPairB + 32 + 8 * ks, ptx::sdesc_sw128(row), id, 1);
                    mma_bf16(leader, d + 16 * ks, tm + L::kPairB + 8 * ks, ptx::sdesc_sw128(row + kTile), id, 1);
                    if (terms == 3) {
                        mma_bf16(leader, d + 16 * ks, tm + L::kPairB + 32 + 8 * ks, ptx::sdesc_sw128(row + kTile), id, 1);
                        mma_bf16(leader, d + 16 * ks, tm + L::kPairB + 8 * ks, ptx::sdesc_sw128(row + 2 * kTile), id, 1);
                    }
                }
            };
            auto times_state = [&](uint32_t d, uint32_t rows, int half) {  // d (+)= (rows S0)^T, 64 of its columns
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = half * 4 + i;
                    const uint64_t bd = ptx::sdesc_sw128(rows + half * 2 * kTile + i * 32);
                    mma_bf16(leader, d, tm + L::kPairS + 8 * j, bd, kRows, j > 0);
                    mma_bf16(leader, d, tm + L::kPairS + N / 2 + 8 * j, bd, kRows, 1);
                }
            };
            wait(kFull0 + (c & 1), c >> 1);
#pragma unroll
            for (int half = 0; half < L::kHalves; ++half) {
                if (half == 0) ptx::named_sync<kPairs, kHalfThreads>();
                else ptx::named_sync<kPairs + 1, kHalfThreads>();
                ptx::tc_fence_after_sync();
                times_state(tm + L::kX, kq, half);
            }
            commit(leader, bar0 + 8 * kXDone);

            ptx::named_sync<kResidual, L::kWorkers + 32>();
            ptx::tc_fence_after_sync();
            lower(tm + L::kX, th, 3, 0);
            commit(leader, bar0 + 8 * kErrDone);
            if (!kStates) {
                if (c > 0) ptx::named_sync<kOutRead, L::kOut + 32>();
                ptx::tc_fence_after_sync();
#pragma unroll
                for (int half = 0; half < L::kHalves; ++half) times_state(tm + L::kO, kq + kTile, half);
                commit(leader, bar0 + 8 * kODone);
            }

            ptx::named_sync<kUpdate, L::kWorkers + 32>();
            ptx::tc_fence_after_sync();
#pragma unroll
            for (int half = 0; half < L::kHalves; ++half) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint64_t bd = sdesc_across(kq + half * 2 * kTile + ks * 16 * 128, 2 * kTile);
                    mma_bf16(leader, tm + L::kS + half * 64, tm + L::kPairC + 8 * ks, bd, kAcross, 1);
                    mma_bf16(leader, tm + L::kS + half * 64, tm + L::kPairC + 32 + 8 * ks, bd, kAcross, 1);
                }
                commit(leader, bar0 + 8 * (kS0Done + half));
            }
            if (kStates) {
                commit(leader, bar0 + 8 * (kDone0 + (c & 1)));
            } else {
                ptx::named_sync<kOutputs, L::kWorkers + L::kOut + 32>();
                ptx::tc_fence_after_sync();
                lower(tm + L::kO, ph, 2, 1);
                commit(leader, bar0 + 8 * (kDone0 + (c & 1)));
            }
        }
        if (kStates)  // nobody else waits for the last chunks': their arrivals must not find another CTA's memory
            for (int c = max(n_chunks - 2, 0); c < n_chunks; ++c) wait_done(c);
        ptx::named_sync<kLast, L::kWorkers + kOuts + 32>();  // the last of it has been read
        ptx::tc_fence_after_sync();
        ptx::tmem_dealloc(tm, 512);
        return;
    }

    const int v = (warp & 3) * 32 + lane;  // this thread's row: a value column of the head
    const uint32_t tl = tm + (static_cast<uint32_t>((warp & 3) * 32) << 16);

    if (kMode == kStateMode && warp >= L::kOutWarp) return;
    if (kKeep && warp >= L::kOutWarp) {  // what the gradients need goes out beside the chain
        const bool first = warp == L::kOutWarp && lane == 0;
#pragma unroll 1
        for (int c = 0; c < n_chunks; ++c) {
            unsigned char *kept = keep.at((slot0 + c) * p.Hv + h, N);
            ptx::named_sync<kOutputs, L::kWorkers + L::kOut>();  // S in pairs
            ptx::tc_fence_after_sync();
            keep_pairs<N, kOutOnly>(tl + L::kPairS, smem + St::kOutAt, kept + gdr_off_state(), kept + gdr_off_state() + 2 * N * N, v, first);
            if (first) ptx::bulk_wait_read<0>();  // the store before has read the staging rows
            ptx::named_sync<kOutOnly, L::kOut>();
            wait(kErrDone, c);
#pragma unroll 1
            for (int part = 0; part < C; part += 32) {
                float x[32];
                uint32_t hi[16], lo[16];
                tm_ld<32>(tl + L::kX + part, x);
                split_row<32>(x, hi, lo);
                put_column<16>(smem + St::kOutAt, v, part, hi);
                put_column<16>(smem + St::kOutAt + C * N * 2, v, part, lo);
            }
            ptx::tc_fence_before_sync();
            if (c + 1 < n_chunks) ptx::named_arrive<kOutRead, L::kWorkers + L::kOut>();
            ptx::fence_proxy_async_smem();
            ptx::named_sync<kOutOnly, L::kOut>();
            if (first) {
                ptx::bulk_store(kept + gdr_off_err(N), base + St::kOutAt, 2 * C * N * 2);
                ptx::bulk_commit();
            }
        }
        if (first) ptx::bulk_wait<0>();
        ptx::named_arrive<kLast, L::kWorkers + kOuts + 32>();
        return;
    }
    if (!kStates && warp >= L::kOutWarp) {
#pragma unroll 1
        for (int c = 0; c < n_chunks; ++c) {
            const float *vec = vec_of(c);
            const int t0 = bos + c * C;
            wait(kFull0 + (c & 1), c >> 1);
            wait(kODone, c);
#pragma unroll
            for (int part = 0; part < C; part += 32) {
                float x[32];
                tm_ld<32>(tl + L::kO + part, x);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 d = *reinterpret_cast<const float4 *>(vec + part + i);
                    x[i] *= d.x * p.scale; x[i + 1] *= d.y * p.scale; x[i + 2] *= d.z * p.scale; x[i + 3] *= d.w * p.scale;
                }
                tm_stf<32>(tl + L::kO + part, x);
            }
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            ptx::named_arrive<kOutputs, L::kWorkers + L::kOut + 32>();

            const bool whole = t0 + C <= eos;
            const bool first = warp == L::kOutWarp && lane == 0;
            if (first) ptx::bulk_wait_read<0>();  // the store before has read the staging rows
            ptx::named_sync<kOutOnly, L::kOut>();
            wait_done(c);
#pragma unroll
            for (int part = 0; part < C; part += 32) {
                float x[32];
                tm_ld<32>(tl + L::kO + part, x);
                if (part == 32 && c + 1 < n_chunks) {
                    ptx::tc_fence_before_sync();
                    ptx::named_arrive<kOutRead, L::kOut + 32>();
                }
                if (whole) {
                    if (p.o_dtype == WKV7_BF16) {
                        __nv_bfloat16 *row = reinterpret_cast<__nv_bfloat16 *>(smem + St::kOutAt) + part * N + v;
#pragma unroll
                        for (int i = 0; i < 32; ++i) row[i * N] = __float2bfloat16_rn(x[i]);
                    } else {
                        float *row = reinterpret_cast<float *>(smem + St::kOutAt) + part * N + v;
#pragma unroll
                        for (int i = 0; i < 32; ++i) row[i * N] = x[i];
                    }
                } else {
                    const long long at = (static_cast<long long>(t0 + part) * p.Hv + h) * N + v, step = static_cast<long long>(p.Hv) * N;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (t0 + part + i < eos) {
                            if (p.o_dtype == WKV7_BF16) static_cast<__nv_bfloat16 *>(p.o)[at + i * step] = __float2bfloat16_rn(x[i]);
                            else static_cast<float *>(p.o)[at + i * step] = x[i];
                        }
                }
            }
            if (whole) {
                ptx::fence_proxy_async_smem();
                ptx::named_sync<kOutOnly, L::kOut>();
                if (first) {
                    ptx::tma_store_2d(&maps.o, h * N, t0, base + St::kOutAt);
                    ptx::bulk_commit();
                }
            }
        }
        if (warp == L::kOutWarp && lane == 0) ptx::bulk_wait<0>();
        ptx::tc_fence_before_sync();
        ptx::named_arrive<kLast, L::kWorkers + kOuts + 32>();
        return;
    }
    if (!L::worker(warp)) return;

    const int wt = L::index(warp, lane), cg = warp >> 2;
    const int k0 = cg * L::kCols, tk0 = cg * L::kTok, half = k0 / 64;
    // S^T: row v, columns k
#pragma unroll 1
    for (int part = 0; part < L::kCols; part += L::kPart) {
        float x[L::kPart];
#pragma unroll
        for (int i = 0; i < L::kPart; ++i)
            x[i] = start(k0 + part + i, v);
        tm_stf<L::kPart>(tl + L::kS + k0 + part, x);
    }
    ptx::tmem_wait_st();

    // (the loop over chunks is kept rolled: the warps' code shares one instruction cache)
#pragma unroll 1
    for (int c = 0; c < n_chunks; ++c) {
        const uint32_t stage = (c & 1) * St::kBytes;
        const float *vec = vec_of(c);
        wait(kFull0 + (c & 1), c >> 1);
        const int len = eos - (bos + c * C);
        if (len < C) {  // rows behind the sequence are another one's: zeros instead
            const uint4 z = make_uint4(0, 0, 0, 0);
            for (int i = len * (N / 8) + wt; i < C * (N / 8); i += L::kWorkers) {
                const int row = i / (N / 8), col = (i % (N / 8)) * 8;
                *reinterpret_cast<uint4 *>(smem + stage + St::kKQ + tile_off<2 * C>(row, col)) = z;
                if (!kStates) *reinterpret_cast<uint4 *>(smem + stage + St::kKQ + tile_off<2 * C>(C + row, col)) = z;
                *reinterpret_cast<uint4 *>(smem + stage + St::kV + (row * N + col) * 2) = z;
            }
            ptx::fence_proxy_async_smem();
            ptx::named_sync<kTail, L::kWorkers>();
        }
        const float dc = vec[C - 1];
        if (c > 0) wait(kS0Done + half, c - 1);
        if (kKeep && c > 0) {  // the pairs and err of the chunk before have been read
            ptx::named_sync<kOutRead, L::kWorkers + L::kOut>();
            ptx::tc_fence_after_sync();
        }
        constexpr int kParts = L::kCols / L::kPart;
        float x0[L::kCols];
        tm_ld<L::kCols>(tl + L::kS + k0, x0);
        auto cols = [&](int part) -> float (&)[L::kPart] { return *reinterpret_cast<float (*)[L::kPart]>(x0 + part * L::kPart); };
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
            uint32_t hi[L::kPart / 2], lo[L::kPart / 2];
            const int at = (k0 + part * L::kPart) / 2;
            split_row<L::kPart>(cols(part), hi, lo);
            tm_st<L::kPart / 2>(tl + L::kPairS + at, hi);
            tm_st<L::kPart / 2>(tl + L::kPairS + N / 2 + at, lo);
        }
        ptx::tmem_wait_st();
        ptx::tc_fence_before_sync();
        if (half == 0) ptx::named_arrive<kPairs, kHalfThreads>();
        else ptx::named_arrive<kPairs + 1, kHalfThreads>();
        if (kKeep) ptx::named_arrive<kOutputs, L::kWorkers + L::kOut>();
#pragma unroll
        for (int part = 0; part < kParts; ++part) {  // d_C S beside the products with the pairs
#pragma unroll
            for (int i = part * L::kPart; i < (part + 1) * L::kPart; i += 2) mul2(x0[i], x0[i + 1], dc);
            tm_stf<L::kPart>(tl + L::kS + k0 + part * L::kPart, cols(part));
        }

        const __nv_bfloat16 *vt = reinterpret_cast<const __nv_bfloat16 *>(smem + stage + St::kV) + tk0 * N + v;
        float r[L::kTok], x[L::kTok];
        uint32_t hi[L::kTok / 2], lo[L::kTok / 2];
#pragma unroll
        for (int i = 0; i < L::kTok; ++i) r[i] = __bfloat162float(vt[i * N]);
        if (kMode == kStateMode && identity) {
#pragma unroll
            for (int i = 0; i < L::kTok; ++i) r[i] = 0.f;
        }
        wait(kXDone, c);
        tm_ld<L::kTok>(tl + L::kX + tk0, x);
#pragma unroll
        for (int i = 0; i < L::kTok; i += 4) {
            const float4 d = *reinterpret_cast<const float4 *>(vec + tk0 + i);
            r[i] = fmaf(-d.x, x[i], r[i]);
            r[i + 1] = fmaf(-d.y, x[i + 1], r[i + 1]);
            r[i + 2] = fmaf(-d.z, x[i + 2], r[i + 2]);
            r[i + 3] = fmaf(-d.w, x[i + 3], r[i + 3]);
        }
        split_row<L::kTok>(r, hi, lo);
        tm_st<L::kTok / 2>(tl + L::kPairB + tk0 / 2, hi);
        tm_st<L::kTok / 2>(tl + L::kPairB + 32 + tk0 / 2, lo);
        ptx::tmem_wait_st();
        ptx::tc_fence_before_sync();
        ptx::named_arrive<kResidual, L::kWorkers + 32>();

        wait(kErrDone, c);
        tm_ld<L::kTok>(tl + L::kX + tk0, x);
#pragma unroll
        for (int i = 0; i < L::kTok; i += 4) {
            const float4 e = *reinterpret_cast<const float4 *>(vec + C + tk0 + i);
            r[i] = e.x * x[i]; r[i + 1] = e.y * x[i + 1]; r[i + 2] = e.z * x[i + 2]; r[i + 3] = e.w * x[i + 3];
        }
        split_row<L::kTok>(r, hi, lo);
        tm_st<L::kTok / 2>(tl + L::kPairC + tk0 / 2, hi);
        tm_st<L::kTok / 2>(tl + L::kPairC + 32 + tk0 / 2, lo);
        ptx::tmem_wait_st();
        ptx::tc_fence_before_sync();
        ptx::named_arrive<kUpdate, L::kWorkers + 32>();

        if (!kStates) {
            split_row<L::kTok>(x, hi, lo);
            tm_st<L::kTok / 2>(tl + L::kPairB + tk0 / 2, hi);
            tm_st<L::kTok / 2>(tl + L::kPairB + 32 + tk0 / 2, lo);
            ptx::tmem_wait_st();
            ptx::tc_fence_before_sync();
            ptx::named_arrive<kOutputs, L::kWorkers + L::kOut + 32>();
        }
        // P err reads pair B until kDone; the next chunk's r is written behind its kXDone, which
        // one thread commits after it
    }
    wait(kS0Done + half, n_chunks - 1);
    if (to) {
#pragma unroll 1
        for (int part = 0; part < L::kCols; part += L::kPart) {
            float x[L::kPart];
            tm_ld<L::kPart>(tl + L::kS + k0 + part, x);
#pragma unroll
            for (int i = 0; i < L::kPart; ++i)
                st_state(to, to_type, to_at + static_cast<long long>(k0 + part + i) * N + v, x[i]);
        }
    }
    ptx::tc_fence_before_sync();
    ptx::named_arrive<kLast, L::kWorkers + kOuts + 32>();
}

}  // namespace forward
}  // namespace gdr
}  // namespace wkv7
