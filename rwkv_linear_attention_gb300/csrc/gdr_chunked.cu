// Chunked prefill of the gated delta rule (wkv7_gdr_prefill with bf16 inputs): the chains of
// gdr_chain.cuh, over whole sequences or segments of them.
//
// Measured: 8 x 4096 tokens, 32 heads of 128, in 293 us (256 chains, 152 at a time, 64 chunks of
// 2.3 us: the three products on the chain are 0.9 of it, the hand-overs between threads and MMAs
// the rest; with That in two terms instead of three 269 us); 30,000 tokens in ten sequences, 40 heads of
// 64, in 250 us.  Before, with the state in the registers of warps that issue mma.sync, the first took 776
// us; with the chunk's matrices formed inside the chain's CTA, 600 us for both where this and
// gdr_prep.cu then took 410 (the code no longer fits the instruction cache).
#include <algorithm>

#include "gdr_chain.cuh"

namespace wkv7 {
namespace gdr {

namespace {
using EncodeTiledFn = decltype(&cuTensorMapEncodeTiled);

EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q);
        return e == cudaSuccess && q == cudaDriverEntryPointSuccess ? reinterpret_cast<EncodeTiledFn>(ptr) : nullptr;
    }();
    return fn;
}

bool make_map(CUtensorMap *map, const void *x, bool bf16, int T_total, long long row, uint32_t cols, CUtensorMapSwizzle swizzle) {
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(row), static_cast<cuuint64_t>(T_total)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(row) * (bf16 ? 2 : 4)};
    const cuuint32_t box[2] = {cols, C}, step[2] = {1, 1};
    return enc(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<void *>(x), dims,
               strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
}  // namespace

bool make_tile_map(CUtensorMap *map, const void *x, int T_total, int heads, int N) {
    return make_map(map, x, true, T_total, static_cast<long long>(heads) * N, 64, CU_TENSOR_MAP_SWIZZLE_128B);
}
bool make_plain_map(CUtensorMap *map, const void *x, bool bf16, int T_total, int heads, int N) {
    return make_map(map, x, bf16, T_total, static_cast<long long>(heads) * N, N, CU_TENSOR_MAP_SWIZZLE_NONE);
}

}  // namespace gdr

namespace {

using namespace gdr;
using namespace gdr::forward;

constexpr int kMaxOrdered = 4096;  // sequences that launch_prefill_order sorts

template <int N, Mode kMode>
__global__ void __launch_bounds__(Chain<N>::kWarps * 32, N == 128 ? 1 : 0)
wkv7_gdr_prefill_chunked_kernel(const GdrPrefillArgs p, const __grid_constant__ GdrMaps maps,
                                const unsigned char *__restrict__ prep, const int32_t *__restrict__ order, const Segments seg) {
    chain<N, kMode>(p, maps, prep, order, GdrChainStore{nullptr}, seg);
}

// The states that segments 2 .. start from: start(s + 1) = A_s start(s) + S_part_s, 32 columns a CTA.
// fp32 throughout; a few microseconds a segment (a thread: 16 columns of one row, N products each).
template <int N>
__global__ void __launch_bounds__(2 * N)
gdr_segment_chain_kernel(const Segments seg, const void *initial_state, wkv7_dtype state_dtype) {
    __shared__ __align__(16) float S[N][36];
    const int tid = threadIdx.x, k = tid >> 1, c = (tid & 1) * 16, v0 = blockIdx.y * 32;
    const long long pair = blockIdx.x;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    if (initial_state) {
        float *copy = seg.start(pair, 0, N * N) + k * N + v0 + c, x[16];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 y = load_state4(initial_state, state_dtype, pair * (N * N) + k * N + v0 + c + i);
            x[i] = y.x; x[i + 1] = y.y; x[i + 2] = y.z; x[i + 3] = y.w;
        }
#pragma unroll
        for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(copy + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    }
    const float *first = seg.start(pair, 1, N * N);
#pragma unroll
    for (int i = 0; i < 16; i += 4) *reinterpret_cast<float4 *>(&S[k][c + i]) = *reinterpret_cast<const float4 *>(first + k * N + v0 + c + i);
    __syncthreads();
    for (int s = 1; s + 1 < seg.count; ++s) {
        const float *part = seg.part(pair, s, N * N) + k * N + v0 + c;
        const float *A = seg.transfer(pair, s, N * N) + k * N;
        float acc[16];
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            const float4 y = *reinterpret_cast<const float4 *>(part + i);
            acc[i] = y.x; acc[i + 1] = y.y; acc[i + 2] = y.z; acc[i + 3] = y.w;
        }
#pragma unroll 8
        for (int j = 0; j < N; j += 4) {
            const float4 a4 = *reinterpret_cast<const float4 *>(A + j);
            const float a[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
            for (int m = 0; m < 4; ++m)
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    const float4 x = *reinterpret_cast<const float4 *>(&S[j + m][c + i]);
                    acc[i] = fmaf(a[m], x.x, acc[i]);
                    acc[i + 1] = fmaf(a[m], x.y, acc[i + 1]);
                    acc[i + 2] = fmaf(a[m], x.z, acc[i + 2]);
                    acc[i + 3] = fmaf(a[m], x.w, acc[i + 3]);
                }
        }
        __syncthreads();
        float *out = seg.start(pair, s + 1, N * N) + k * N + v0 + c;
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4 *>(out + i) = *reinterpret_cast<float4 *>(&S[k][c + i]) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
        __syncthreads();
    }
}

constexpr int kSms = 152;

// Segments per sequence.  With n chunks a sequence and both passes' chains on the SMs at once, a
// segmented call takes n / count chunk steps twice (1.75 us without outputs, 2.3 with them) instead
// of n once, and about 15 us for the small kernel and two more launches: 48 chunks in 8 segments
// take 22 + 15 us instead of 86, 24 in 3 take 29 + 15 instead of 43.  If one segment more would
// leave few of the first pass's runs without an SM, the two runs of the last segment that it runs
// are made half as long, come last, and share: 32768 tokens with 32 heads of 128 in 732 us
// instead of 805 in three equal segments (both measured when a step took 1.7 and 2.1).  The sequences'
// mean length decides, which host and device know alike: one long sequence among short ones is not cut.
Segments segments(int num_seqs, int T_total, int Hv) {
    const long long pairs = static_cast<long long>(num_seqs) * Hv;
    if (pairs == 0) return {1, false, nullptr};
    const long long most = std::min(T_total / C / num_seqs / 6, 16);
    const long long count = std::min(std::min((kSms / pairs + 3) / 2, kSms / pairs), most);
    if (count < 3) return {1, false, nullptr};
    const long long over = (2 * count - 1) * pairs - kSms;  // runs without an SM, with count + 1 segments
    if (count < most && (count + 1) * pairs <= kSms && over > 0 && over <= pairs) return {static_cast<int>(count) + 1, true, nullptr};
    return {static_cast<int>(count), false, nullptr};
}

template <int N, Mode kMode>
cudaError_t chains(const GdrPrefillArgs &p, const GdrMaps &maps, const unsigned char *prep, const int32_t *order,
                   Segments seg, cudaStream_t stream) {
    static std::atomic<unsigned long long> allowed{0};
    constexpr int kSmem = Stage<N>::kSmem;
    static_assert(kSmem <= 226 * 1024, "two stages and the output rows fit one SM");
    const cudaError_t e = gdr_allow_smem(reinterpret_cast<const void *>(wkv7_gdr_prefill_chunked_kernel<N, kMode>), kSmem, allowed);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(p.num_seqs) * static_cast<unsigned>(p.Hv),
                    seg.count == 1 ? 1 : kMode == kStateMode ? seg.first_pass_runs() : seg.count);
    return gdr_launch(wkv7_gdr_prefill_chunked_kernel<N, kMode>, grid, Chain<N>::kWarps * 32, kSmem, stream, p.T_total > 0,
                             p, maps, prep, order, seg);
}

template <int N>
cudaError_t prefill(const GdrPrefillArgs &p, const GdrMaps &maps, const unsigned char *prep, const int32_t *order, Segments seg, cudaStream_t stream) {
    if (seg.count > 1) {
        cudaError_t e = chains<N, kStateMode>(p, maps, prep, order, seg, stream);
        if (e != cudaSuccess) return e;
        e = gdr_launch(gdr_segment_chain_kernel<N>, dim3(static_cast<unsigned>(p.num_seqs) * static_cast<unsigned>(p.Hv), N / 32),
                              2 * N, 0, stream, true, seg, p.initial_state, p.state_dtype);
        if (e != cudaSuccess) return e;
    }
    return chains<N, kOutputsMode>(p, maps, prep, order, seg, stream);
}

}  // namespace

bool gdr_forward_maps(GdrMaps *maps, const GdrPrefillArgs &p) {
    if (p.T_total == 0) return true;
    return make_tile_map(&maps->k, p.k, p.T_total, p.Hk, p.N) && make_tile_map(&maps->q, p.q, p.T_total, p.Hk, p.N) &&
           make_plain_map(&maps->v, p.v, true, p.T_total, p.Hv, p.N) &&
           (!p.o || make_plain_map(&maps->o, p.o, p.o_dtype == WKV7_BF16, p.T_total, p.Hv, p.N));
}

size_t gdr_order_bytes(int num_seqs) {
    return num_seqs > kGdrRanked && num_seqs <= kMaxOrdered ? (static_cast<size_t>(num_seqs) * 4 + 1023) / 1024 * 1024 : 0;
}

cudaError_t launch_gdr_order(const GdrPrefillArgs &p, void *workspace, int32_t **order, cudaStream_t stream) {
    *order = nullptr;
    if (!gdr_order_bytes(p.num_seqs) || p.T_total == 0) return cudaSuccess;
    *order = static_cast<int32_t *>(workspace);
    PrefillArgs a = {};
    a.num_seqs = p.num_seqs;
    a.cu_seqlens = p.cu_seqlens;
    return launch_prefill_order(a, *order, stream);
}

namespace {
size_t segment_bytes(int num_seqs, int T_total, int Hv, int N) {
    const Segments seg = segments(num_seqs, T_total, Hv);
    return seg.count == 1 ? 0 : static_cast<size_t>(num_seqs) * Hv * seg.slots() * N * N * sizeof(float);
}
}  // namespace

size_t gdr_chunked_workspace_bytes(int num_seqs, int T_total, int Hv, int N) {
    return gdr_order_bytes(num_seqs) + 112 + gdr_prep_bytes(num_seqs, T_total, Hv) + segment_bytes(num_seqs, T_total, Hv, N);
}

cudaError_t launch_gdr_prefill_chunked(const GdrPrefillArgs &p, void *workspace, cudaStream_t s) {
    unsigned char *prep = gdr_behind_order(workspace, p.num_seqs);
    Segments seg = segments(p.num_seqs, p.T_total, p.Hv);
    seg.scratch = reinterpret_cast<float *>(prep + gdr_prep_bytes(p.num_seqs, p.T_total, p.Hv));
    GdrMaps maps = {};
    if (!gdr_forward_maps(&maps, p)) return cudaErrorInvalidValue;
    int32_t *order;
    cudaError_t e = launch_gdr_order(p, workspace, &order, s);
    if (e == cudaSuccess && p.T_total > 0) e = launch_gdr_prep(p, maps, prep, s);
    if (e != cudaSuccess) return e;
    return p.N == 64 ? prefill<64>(p, maps, prep, order, seg, s) : prefill<128>(p, maps, prep, order, seg, s);
}

}  // namespace wkv7
