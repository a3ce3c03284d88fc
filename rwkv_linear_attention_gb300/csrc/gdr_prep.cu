// The chunk matrices of the gated delta rule (gdr_prep.cuh) for every chunk and value head,
// ahead of the chains.
//
// One CTA of four warps per (chunk, query/key head): the K and Q rows come by TMA, one MMA forms
// their products with K in tensor memory (64 columns), and each value head that shares them takes
// its That and P from those.  The steps of a head are short and follow one another, so latency
// bounds a CTA and several share an SM; together they are bound by what they write (25 KB of
// matrices per chunk and head: the blocks above the diagonal are not written; the chains copy whole
// tiles, but no product of theirs uses those blocks).
//
// Measured: 8 x 4096 tokens, 32 heads of 128 in 177 us, 30,000 tokens with 40 heads of 64 in 230 us
// (0.73 and 0.84 GB through HBM, 4.1 and 3.7 TB/s; That in two terms instead of three: 141 and 197 us).
// Four CTAs an SM instead of five: 246 us in the second case.
#include "gdr_internal.cuh"
#include "gdr_prep.cuh"

namespace wkv7 {
namespace {

using namespace gdr;

constexpr int kThreads = 128;
constexpr int kHeads = 2;  // heads whose vectors are formed at once, one per warp (and 42 KB a CTA: five share an SM)
constexpr uint32_t kMaxPolls = 1u << 17;  // of up to 20 us: seconds

template <int N>
struct Smem {
    static constexpr uint32_t kRows = 0;                       // K rows 0-63, Q rows 64-127, [128][64] blocks
    static constexpr uint32_t kThat = 0;                       // in their place: That's three tiles
    static constexpr uint32_t kDiag = 2 * C * N * 2 > 3 * kTile ? 2 * C * N * 2 : 3 * kTile;
    static constexpr uint32_t kVec = kDiag + 4 * 16 * kDiagLd * 4;
    static constexpr uint32_t kBytes = kVec + kHeads * kVecFloats * 4;
};

template <int N>
__global__ void __launch_bounds__(kThreads, 5)
gdr_prep_kernel(const GdrPrefillArgs p, const __grid_constant__ GdrMaps maps, unsigned char *__restrict__ prep) {
    using M = Smem<N>;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(8) unsigned long long bars[2];  // rows, products
    __shared__ uint32_t s_tmem;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int slot = blockIdx.x, hk = blockIdx.y, rep = p.Hv / p.Hk;
    const int b = gdr_find_seq(p.cu_seqlens, p.num_seqs, slot, lane);
    int bos, eos;
    if (!gdr_seq_bounds(p.cu_seqlens, p.num_seqs, p.T_total, b, bos, eos)) return;  // reported by the chain
    const int chunk = slot - ((bos >> 6) + b);
    if (chunk < 0 || chunk >= (eos - bos + C - 1) / C) return;
    const int t0 = bos + chunk * C, t1 = min(eos, t0 + C), len = t1 - t0;

    const uint32_t base = ptx::smem_addr(smem), rows_bar = ptx::smem_addr(&bars[0]), gram_bar = ptx::smem_addr(&bars[1]);
    if (warp == 0) {
        if (lane == 0) {
            ptx::mbar_init(rows_bar, 1);
            ptx::mbar_init(gram_bar, 1);
            ptx::fence_mbar_init();
            ptx::mbar_arrive_expect_tx(rows_bar, 2 * C * N * 2);
#pragma unroll
            for (int j = 0; j < N / 64; ++j) {
                ptx::tma_load_2d(base + M::kRows + j * 2 * kTile, &maps.k, hk * N + j * 64, t0, rows_bar);
                ptx::tma_load_2d(base + M::kRows + j * 2 * kTile + kTile, &maps.q, hk * N + j * 64, t0, rows_bar);
            }
        }
        __syncwarp();
        ptx::tmem_alloc(ptx::smem_addr(&s_tmem), 64);
    }
    float *vecs = reinterpret_cast<float *>(smem + M::kVec);
    auto vectors = [&](int r0) {
        if (warp < kHeads && r0 + warp < rep) chunk_vectors(p, hk * rep + r0 + warp, t0, t1, lane, vecs + warp * kVecFloats);
    };
    vectors(0);
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    ptx::grid_dep_launch();
    bool ok = wait_phase(rows_bar, 0, kMaxPolls);
    if (len < C) {  // rows behind the sequence are another one's: zeros instead
        const uint4 z = make_uint4(0, 0, 0, 0);
        for (int i = len * (N / 8) + tid; i < C * (N / 8); i += kThreads) {
            const int row = i / (N / 8), col = (i % (N / 8)) * 8;
            *reinterpret_cast<uint4 *>(smem + M::kRows + tile_off<2 * C>(row, col)) = z;
            *reinterpret_cast<uint4 *>(smem + M::kRows + tile_off<2 * C>(C + row, col)) = z;
        }
        ptx::fence_proxy_async_smem();
        __syncthreads();
    }
    const uint32_t tm = s_tmem;
    if (warp == 0) {
        const uint32_t leader = elect_lane();
#pragma unroll
        for (int j = 0; j < N / 16; ++j) {
            const uint64_t bd = ptx::sdesc_sw128(base + M::kRows + (j >> 2) * 2 * kTile + (j & 3) * 32);
            mma_bf16_ss(leader, tm, bd, bd, idesc_bf16(128, 64, false), j > 0);
        }
        commit(leader, gram_bar);
    }
    ok = wait_phase(gram_bar, 0, kMaxPolls) && ok;
    ptx::tc_fence_after_sync();
    if (!ok && lane == 0) report(p.status, kDevTimeout);

#pragma unroll 1
    for (int r = 0; r < rep; ++r) {
        const int w = r % kHeads;
        __syncthreads();  // the scratch, and before the first head the rows, have been read
        if (r > 0 && w == 0) {
            vectors(r);
            __syncthreads();
        }
        float *vec = vecs + w * kVecFloats;
        unsigned char *out = prep + (static_cast<long long>(slot) * p.Hv + hk * rep + r) * kGdrPrepBytes;
        chunk_matrices<1>(smem, tm, M::kThat, out, reinterpret_cast<float *>(smem + M::kDiag), vec, p.scale, warp, lane);
        if (tid < kVecKept / 4)
            reinterpret_cast<float4 *>(out + kGdrPrepVec)[tid] = reinterpret_cast<const float4 *>(vec)[tid];
        __syncthreads();
#pragma unroll 4
        for (int i = tid; i < 3 * C * 8; i += kThreads) {  // That's blocks on and below the diagonal
            const int row = (i >> 3) & (C - 1);
            if ((((i & 7) ^ (row & 7)) >> 1) <= (row >> 4))
                *reinterpret_cast<uint4 *>(out + kGdrPrepThat + i * 16) = *reinterpret_cast<const uint4 *>(smem + M::kThat + i * 16);
        }
    }
    ptx::tc_fence_before_sync();
    __syncthreads();
    ptx::tc_fence_after_sync();
    if (warp == 0) ptx::tmem_dealloc(tm, 64);
}

template <int N>
cudaError_t run(const GdrPrefillArgs &p, const GdrMaps &maps, unsigned char *prep, cudaStream_t stream) {
    static std::atomic<unsigned long long> allowed{0};
    constexpr int kSmem = Smem<N>::kBytes;
    const cudaError_t e = gdr_allow_smem(reinterpret_cast<const void *>(gdr_prep_kernel<N>), kSmem, allowed);
    if (e != cudaSuccess) return e;
    const dim3 grid(static_cast<unsigned>(gdr_max_slots(p.num_seqs, p.T_total)), p.Hk);
    gdr_prep_kernel<N><<<grid, kThreads, kSmem, stream>>>(p, maps, prep);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_gdr_prep(const GdrPrefillArgs &p, const GdrMaps &maps, unsigned char *prep, cudaStream_t stream) {
    return p.N == 64 ? run<64>(p, maps, prep, stream) : run<128>(p, maps, prep, stream);
}

}  // namespace wkv7
