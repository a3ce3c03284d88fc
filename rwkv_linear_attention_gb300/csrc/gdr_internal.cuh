// Internal declarations of the gated delta rule (wkv7_gdr_*) and of draft
// acceptance (wkv7_verify_accept).  Not part of the C ABI (include/wkv7.h).
#pragma once

#include <cuda.h>

#include <atomic>

#include "wkv7_internal.cuh"

namespace wkv7 {

// The current device's status word, and the record of a CUDA error (wkv7_api.cu).
wkv7_status device_status_word(unsigned **out);
wkv7_status record_cuda_error(cudaError_t e);

constexpr int kGdrChunk = 64;  // tokens per chunk of the chunked kernels

// A log-decay below this is taken as this: exp of it is already exactly 0 in fp32, and
// sums of a chunk's decays stay exact integers plus a fraction.  NaN passes through.
constexpr float kGdrMinLogDecay = -10000.f;
__device__ __forceinline__ float gdr_clamp_decay(float g) { return g < kGdrMinLogDecay ? kGdrMinLogDecay : g; }

// Allow `kernel` its dynamic shared memory, once per device (`done`: the kernel's own flags).
inline cudaError_t gdr_allow_smem(const void *kernel, int bytes, std::atomic<unsigned long long> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// Launch a kernel of a call.  With `behind` it may start while the grid of the call's own kernel before
// it still runs, and waits for that one (griddepcontrol.wait) before it reads what the call's kernels
// wrote and before it writes at all; a call's first kernel waits for all of the stream's work, as
// any launch.  A kernel lets the next one come only once its own tensor memory is allocated (a later
// allocation could stand in its way), and the chains that run for states alone not before they end:
// the small kernel behind them would crowd the SMs that are free first.  The backward of six documents
// to 300 tokens took 75 us without and 67 with, prefill of 32768 tokens 726 and 719 (measured when the
// backward's chains still were two launches).
template <typename... Params, typename... Args>
inline cudaError_t gdr_launch(void (*kernel)(Params...), dim3 grid, unsigned threads, int smem, cudaStream_t stream, bool behind,
                              const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = behind ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

struct GdrStepArgs {
    int B, Hk, Hv, N;
    wkv7_dtype x_dtype;      // q, k, v: WKV7_F32 or WKV7_BF16
    const void *q, *k;       // [B, Hk, N]
    const void *v;           // [B, Hv, N]
    const float *g, *beta;   // [B, Hv]
    float scale;
    void *state;             // [B, Hv, N, N] of state_dtype, in place
    wkv7_dtype state_dtype;
    void *o;                 // [B, Hv, N] of o_dtype
    wkv7_dtype o_dtype;
};
cudaError_t launch_gdr_step(const GdrStepArgs &args, cudaStream_t stream);

// The sequence of this rank, the longest first, where a warp can rank them all; else as they come.
// A permutation whatever the offsets hold.
constexpr int kGdrRanked = 32;
__device__ __forceinline__ int gdr_by_length(const int32_t *cu_seqlens, int num_seqs, int rank, int lane) {
    if (num_seqs == 1 || num_seqs > kGdrRanked) return rank;
    const int len = lane < num_seqs ? cu_seqlens[lane + 1] - cu_seqlens[lane] : 0;
    int before = 0;
    for (int i = 0; i < num_seqs; ++i) {
        const int l = __shfl_sync(0xffffffffu, len, i);
        before += l > len || (l == len && i < lane);
    }
    return __ffs(__ballot_sync(0xffffffffu, lane < num_seqs && before == rank)) - 1;
}

struct GdrPrefillArgs {
    int num_seqs, T_total, Hk, Hv, N;
    const int32_t *cu_seqlens;  // device [num_seqs + 1]
    wkv7_dtype x_dtype;
    const void *q, *k, *v;
    const float *g, *beta;
    float scale;
    const void *initial_state;  // nullable
    void *final_state;          // nullable
    wkv7_dtype state_dtype;
    void *o;
    wkv7_dtype o_dtype;
    unsigned *status;
    const int32_t *cu_seqlens_host;  // nullable; only for the choice of a split
};
cudaError_t launch_gdr_prefill_scan(const GdrPrefillArgs &args, cudaStream_t stream);

// The chunked kernels (bf16 inputs).
//
// Chunk slots.  Sequence b's chunks have the slots cu[b] / 64 + b, + 1, ..: a sequence of
// n tokens from token x takes ceil(n / 64) <= (x + n) / 64 - x / 64 + 1 slots, so the ranges
// are disjoint, end at T / 64 + num_seqs, and need no scan over the sequences.
inline long long gdr_max_slots(int num_seqs, int T_total) { return static_cast<long long>(T_total) / kGdrChunk + num_seqs; }

// What the chunk kernels share per (slot, value head), written by gdr_prep.cu:
//   [P hi][P lo][That in three terms]  bf16 tiles [64][64] (gdr_mma.cuh)
//   d[64], e[64], beta[64], gam as integer [64] and fraction [64] of log2,
//   e without beta [64]                fp32
constexpr int kGdrPrepThat = 2 * 8192, kGdrPrepVec = 5 * 8192, kGdrPrepBytes = kGdrPrepVec + 2048;
inline size_t gdr_prep_bytes(int num_seqs, int T_total, int Hv) {
    return static_cast<size_t>(gdr_max_slots(num_seqs, T_total)) * Hv * kGdrPrepBytes;
}
// The tensors of a call as the kernels' copies see them (each encoded once a call): rows of 64
// tokens, in swizzled 64-column tiles (k, q, d_o, dv) or plain (v; o, or the backward's dv).
struct GdrMaps {
    CUtensorMap k, q, v, o, d_o, dv;
};
bool gdr_forward_maps(GdrMaps *maps, const GdrPrefillArgs &args);
cudaError_t launch_gdr_prep(const GdrPrefillArgs &args, const GdrMaps &maps, unsigned char *prep, cudaStream_t stream);

// Bytes of workspace, and the call itself.
size_t gdr_chunked_workspace_bytes(int num_seqs, int T_total, int Hv, int N);
cudaError_t launch_gdr_prefill_chunked(const GdrPrefillArgs &args, void *workspace, cudaStream_t stream);

// Backward.
struct GdrBackwardArgs {
    GdrPrefillArgs f;       // the forward call's inputs (states fp32, no outputs)
    const void *d_o;        // [T_total, Hv, N] bf16
    const float *d_final_state;  // nullable
    void *dq, *dk, *dv;     // bf16
    float *dg, *dbeta;      // [T_total, Hv]
    float *d_initial_state;  // nullable
};
// What the chains leave per (slot, value head) for the gradients, pairs of bf16 tiles: the state
// before the chunk and the adjoint behind it ([v][k]), err ([token][v]), and the low tile of dv
// ([token][v]; the high one is dv itself).
inline size_t gdr_chain_bytes(int N) { return 8u * N * N + 8u * N * kGdrChunk; }
struct GdrChainStore {
    unsigned char *base;  // null: nothing is kept
    __device__ __forceinline__ unsigned char *at(long long i, int N) const {
        return base + i * (8ll * N * N + 8ll * N * kGdrChunk);
    }
};
constexpr long long gdr_off_state() { return 0; }
constexpr long long gdr_off_adjoint(int N) { return 4ll * N * N; }
constexpr long long gdr_off_err(int N) { return 8ll * N * N; }
constexpr long long gdr_off_dv(int N) { return 8ll * N * N + 4ll * N * kGdrChunk; }
// The order of more sequences than a warp ranks, longest first, at the workspace's start (else null),
// and what follows it there, on a 128-byte boundary (workspaces need only 16).
size_t gdr_order_bytes(int num_seqs);
inline unsigned char *gdr_behind_order(void *workspace, int num_seqs) {
    return reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(workspace) + gdr_order_bytes(num_seqs) + 127) & ~static_cast<uintptr_t>(127));
}
cudaError_t launch_gdr_order(const GdrPrefillArgs &args, void *workspace, int32_t **order, cudaStream_t stream);
size_t gdr_backward_workspace_bytes(int num_seqs, int T_total, int Hv, int N);
cudaError_t launch_gdr_prefill_backward(const GdrBackwardArgs &args, void *workspace, cudaStream_t stream);

// Token range of sequence b; false (and a report) where cu_seqlens is malformed there.
__device__ __forceinline__ bool gdr_seq_bounds(const int32_t *cu, int num_seqs, int T_total, int b, int &bos, int &eos) {
    bos = cu[b];
    eos = cu[b + 1];
    return bos >= 0 && eos >= bos && eos <= T_total && (b > 0 || bos == 0) && (b + 1 < num_seqs || eos == T_total);
}

// The sequence whose slots hold `slot`: the last b with cu[b] / 64 + b <= slot, found by a
// whole warp, 32 probes at a time.  Some index in 0 .. num_seqs - 1 where cu is malformed.
__device__ __forceinline__ int gdr_find_seq(const int32_t *cu, int num_seqs, int slot, int lane) {
    int lo = 0, n = num_seqs;
    while (n > 1) {
        const int step = (n + 31) / 32, at = lo + lane * step;
        const bool below = lane * step < n && (static_cast<long long>(cu[at]) >> 6) + at <= slot;
        const int k = max(0, __popc(__ballot_sync(0xffffffffu, below)) - 1);
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo;
}

// Draft acceptance.
struct AcceptArgs {
    int B, K, V;
    const int32_t *draft_tokens;  // [B, K]
    const int32_t *draft_lens;    // [B] or null (all K)
    const float *target_probs;    // [B, K + 1, V]
    const float *draft_probs;     // [B, K, V] or null (each draft certain)
    const float *u_accept;        // [B, K]
    const float *u_sample;        // [B]
    int32_t *accept_len;          // [B]
    int32_t *next_token;          // [B]
    unsigned *status;
};
cudaError_t launch_verify_accept(const AcceptArgs &args, cudaStream_t stream);

// Four consecutive elements of a row of type dt (F32 or BF16), widened to fp32.
template <bool kBf16>
__device__ __forceinline__ float4 gdr_load4(const void *base, long long idx) {
    if (!kBf16) return *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + idx);
    const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + idx);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
}

}  // namespace wkv7
