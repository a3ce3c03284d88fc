// Draft acceptance for a speculative step (wkv7_verify_accept): which drafted tokens a
// verify pass keeps, and the token that follows them, from given random numbers.
//
// Per row, with target distributions p_0 .. p_K (one per position of the verify pass)
// and draft distributions q_0 .. q_{K-1}:
//
//   draft i is kept while u_i q_i(x_i) < p_i(x_i)          (kept with probability min(1, p/q))
//   n = the number of drafts kept before the first refusal
//   weights  m(v) = max(p_n(v) - q_n(v), 0) after a refusal, p_K(v) when all were kept
//   next     = the smallest v with  sum_{j <= v} m(j)  >  u * sum_j m(j)
//
// so the kept tokens and the next one are distributed as the target's own samples.
//
// The answer is a whole number that a rounding can change, so nothing here is rounded
// in 32 bits: u q < p is compared as a 48-bit product in fp64, p - q is kept exactly as
// an fp32 pair (difference and its error), and every sum is such a pair (error-free
// additions, about 46 bits).  fp64 sums would be bound by the fp64 pipe (two lanes a clock
// and SM): with fp64 reductions per segment and an fp64 search, 256 rows of 100003 took
// 185 us and the pipe alone 51; in pairs on the fp32 pipe they take 47
// (4.4 TB/s; the dependent loads before and after the sums are most of the rest).
//
// One cluster of 1 - 8 CTAs per row.  Only row n of p and row n of q are read, once: a
// warp sums segments of 256 consecutive weights (eight per lane of each row, all loads in
// flight together; single-word loads because rows of an odd V share no alignment).  The
// CTA totals meet in distributed shared memory, the one CTA whose range holds the
// threshold finds the segment from its segment sums and reads that segment again (from L2).
#include <cooperative_groups.h>

#include "gdr_internal.cuh"

namespace wkv7 {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kLane = 8;            // weights per lane and segment
constexpr int kSeg = 32 * kLane;    // weights per segment
constexpr int kCtasPerSm = 4;

// An unevaluated sum hi + lo, |lo| <= half a step of hi.
struct Pair {
    float hi, lo;
};

__device__ __forceinline__ Pair add(Pair a, Pair b) {
    const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
    const float err = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
    const float lo = __fadd_rn(err, __fadd_rn(a.lo, b.lo));
    const float hi = __fadd_rn(s, lo);
    return {hi, __fsub_rn(lo, __fsub_rn(hi, s))};
}
__device__ __forceinline__ bool less(Pair a, Pair b) { return a.hi < b.hi || (a.hi == b.hi && a.lo < b.lo); }
__device__ __forceinline__ Pair scale(float u, Pair a) {  // u a
    const float p = __fmul_rn(u, a.hi), e = fmaf(u, a.lo, fmaf(u, a.hi, -p));
    const float hi = __fadd_rn(p, e);
    return {hi, __fsub_rn(e, __fsub_rn(hi, p))};
}
__device__ __forceinline__ Pair times_power(Pair a, float p) { return {a.hi * p, a.lo * p}; }  // p a power of two: exact
__device__ __forceinline__ Pair shfl_xor(Pair a, int m) {
    return {__shfl_xor_sync(0xffffffffu, a.hi, m), __shfl_xor_sync(0xffffffffu, a.lo, m)};
}
// The sum over the warp: the same pair, bit for bit, in every lane (additions of two
// neighbours commute, and all lanes add the same two halves at each level).
__device__ __forceinline__ Pair warp_sum(Pair a) {
#pragma unroll
    for (int off = 16; off; off >>= 1) a = add(a, shfl_xor(a, off));
    return a;
}
// The sum over this lane and the lanes below.
__device__ __forceinline__ Pair warp_scan(Pair a, int lane) {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const Pair o{__shfl_up_sync(0xffffffffu, a.hi, off), __shfl_up_sync(0xffffffffu, a.lo, off)};
        if (lane >= off) a = add(o, a);
    }
    return a;
}

// max(p - q, 0), exactly.  A NaN on either side weighs nothing.
__device__ __forceinline__ Pair weight(float p, float q) {
    const float s = __fsub_rn(p, q), t = __fsub_rn(s, p);
    const float err = __fsub_rn(__fsub_rn(p, __fsub_rn(s, t)), __fadd_rn(q, t));
    const bool pos = p > q;
    return {pos ? s : 0.f, pos ? err : 0.f};
}

// The sum of a lane's weights: the errors of the leading sums are added up, and joined at the end.
__device__ __forceinline__ Pair sum_of(const Pair (&w)[kLane]) {
    float hi = w[0].hi, lo = w[0].lo;
#pragma unroll
    for (int j = 1; j < kLane; ++j) {
        const float s = __fadd_rn(hi, w[j].hi), t = __fsub_rn(s, hi);
        const float err = __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(w[j].hi, t));
        lo = __fadd_rn(lo, __fadd_rn(err, w[j].lo));
        hi = s;
    }
    const float s = __fadd_rn(hi, lo);
    return {s, __fsub_rn(lo, __fsub_rn(s, hi))};
}

struct Row {
    const float *p;   // target row
    const float *q;   // draft row, or null
    int certain;      // q is 1 at this token and 0 elsewhere (-1: nowhere)
    __device__ __forceinline__ float sub(int v) const { return q ? q[v] : (v == certain ? 1.f : 0.f); }
};

__global__ void __launch_bounds__(kThreads, kCtasPerSm)
wkv7_verify_accept_kernel(const AcceptArgs a, int segs_per_cta) {
    extern __shared__ Pair seg_sum[];  // [segs_per_cta]
    __shared__ Pair cta_sum[2];        // one per pass: the other CTAs may still read the first
    __shared__ int s_n, s_len;
    cg::cluster_group cluster = cg::this_cluster();
    const int ranks = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
    const long long b = blockIdx.x / ranks;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    // ---- how many drafts are kept
    float u = a.u_sample[b];
    if (warp == 0) {
        int len = a.K;
        if (a.draft_lens) {
            len = a.draft_lens[b];
            if (len < 0 || len > a.K) {
                if (lane == 0 && rank == 0) report(a.status, kDevBounds);
                len = len < 0 ? 0 : a.K;
            }
        }
        bool keep = false;
        if (lane < len) {
            const int x = a.draft_tokens[b * a.K + lane];
            if (x >= 0 && x < a.V) {
                const double p = a.target_probs[(b * (a.K + 1) + lane) * a.V + x];
                const double q = a.draft_probs ? a.draft_probs[(b * a.K + lane) * a.V + x] : 1.f;
                keep = static_cast<double>(a.u_accept[b * a.K + lane]) * q < p;
            } else if (rank == 0) {
                report(a.status, kDevBounds);
            }
        }
        const unsigned kept = __ballot_sync(0xffffffffu, keep);  // lane 31 holds no draft
        if (lane == 0) {
            s_n = __ffs(~kept) - 1;
            s_len = len;
            if (rank == 0) a.accept_len[b] = s_n + 1;
        }
    }
    __syncthreads();
    const int n = s_n;
    Row row{a.target_probs + (b * (a.K + 1) + n) * a.V, nullptr, -1};
    if (n < s_len) {
        if (a.draft_probs) row.q = a.draft_probs + (b * a.K + n) * a.V;
        else row.certain = a.draft_tokens[b * a.K + n];
    }
    u = u > 0.f ? fminf(u, 0x1.fffffep-1f) : 0.f;
    const int first = rank * segs_per_cta * kSeg;  // below V + 8 * 256, V <= 2^24

    for (int pass = 0; pass < 2; ++pass) {  // pass 1: no weight was left, the target's own row
        auto load = [&](int s, float (&p)[kLane], float (&q)[kLane]) {
            const int v0 = first + s * kSeg + lane;
            if (v0 - lane + kSeg <= a.V && (row.q || row.certain < 0)) {
#pragma unroll
                for (int j = 0; j < kLane; ++j) p[j] = row.p[v0 + 32 * j];
#pragma unroll
                for (int j = 0; j < kLane; ++j) q[j] = row.q ? row.q[v0 + 32 * j] : 0.f;
            } else {
#pragma unroll
                for (int j = 0; j < kLane; ++j) {
                    const int v = v0 + 32 * j;
                    const bool in = v < a.V;
                    p[j] = in ? row.p[v] : 0.f;
                    q[j] = in ? row.sub(v) : 0.f;
                }
            }
        };
        float p[kLane], q[kLane];
        if (warp < segs_per_cta) load(warp, p, q);
        for (int s = warp; s < segs_per_cta; s += kWarps) {
            Pair w[kLane];
#pragma unroll
            for (int j = 0; j < kLane; ++j) w[j] = weight(p[j], q[j]);
            if (s + kWarps < segs_per_cta) load(s + kWarps, p, q);  // under way while these are summed
            const Pair sum = warp_sum(sum_of(w));
            if (lane == 0) seg_sum[s] = sum;
        }
        __syncthreads();
        if (warp == 0) {  // this CTA's total, in a fixed order
            Pair sum{0.f, 0.f};
            for (int s = lane; s < segs_per_cta; s += 32) sum = add(sum, seg_sum[s]);
            sum = warp_sum(sum);
            if (lane == 0) cta_sum[pass] = sum;
        }
        cluster.sync();
        Pair total{0.f, 0.f}, before{0.f, 0.f}, upto{0.f, 0.f};
        for (int r = 0; r < ranks; ++r) {
            if (r == rank) before = total;
            total = add(total, *cluster.map_shared_rank(&cta_sum[pass], r));
            if (r == rank) upto = total;
        }
        if (total.hi > 0.f && total.hi < INFINITY) {
            // The threshold and what is compared with it are taken 2^64 times as large where that
            // leaves room: near the smallest fp32 numbers u times the total would round to the
            // total itself, and no sum would pass it.  So enlarged, u total < total holds, and the
            // ranges [before, upto) of the row's CTAs leave no gap: one of them has the threshold.
            const float up = total.hi < 0x1p60f ? 0x1p64f : 1.f;
            const Pair thr = scale(u, times_power(total, up));
            auto past_at = [&](Pair sum) { return less(thr, times_power(sum, up)); };
            if (warp == 0 && !past_at(before) && past_at(upto)) {
                // the first segment whose running sum passes the threshold (rounding may leave
                // it past the last one: then the last with any weight)
                Pair at = before, seg_at = before;
                int seg = -1, last = 0;
                Pair last_at = before;
                for (int s0 = 0; s0 < segs_per_cta && seg < 0; s0 += 32) {
                    const Pair own = s0 + lane < segs_per_cta ? seg_sum[s0 + lane] : Pair{0.f, 0.f};
                    const Pair incl = add(at, warp_scan(own, lane));
                    Pair excl{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
                    if (lane == 0) excl = at;
                    const unsigned past = __ballot_sync(0xffffffffu, own.hi > 0.f && past_at(incl));
                    const unsigned any = __ballot_sync(0xffffffffu, own.hi > 0.f);
                    const int pick = past ? __ffs(past) - 1 : any ? 31 - __clz(any) : 0;
                    const Pair pick_at{__shfl_sync(0xffffffffu, excl.hi, pick), __shfl_sync(0xffffffffu, excl.lo, pick)};
                    if (past) {
                        seg = s0 + pick;
                        seg_at = pick_at;
                    } else if (any) {
                        last = s0 + pick;
                        last_at = pick_at;
                    }
                    at = Pair{__shfl_sync(0xffffffffu, incl.hi, 31), __shfl_sync(0xffffffffu, incl.lo, 31)};
                }
                if (seg < 0) {
                    seg = last;
                    seg_at = last_at;
                }
                // within it: eight consecutive weights per lane
                const int v0 = first + seg * kSeg + lane * kLane;
                Pair w[kLane], own{0.f, 0.f};
#pragma unroll
                for (int j = 0; j < kLane; ++j) {
                    const int v = v0 + j;
                    w[j] = v < a.V ? weight(row.p[v], row.sub(v)) : Pair{0.f, 0.f};
                    own = add(own, w[j]);
                }
                const Pair incl = warp_scan(own, lane);
                Pair c{__shfl_up_sync(0xffffffffu, incl.hi, 1), __shfl_up_sync(0xffffffffu, incl.lo, 1)};
                c = lane == 0 ? seg_at : add(seg_at, c);
                int hit = -1, pos = -1;
#pragma unroll
                for (int j = 0; j < kLane; ++j) {
                    c = add(c, w[j]);
                    if (w[j].hi > 0.f) {
                        pos = v0 + j;
                        if (hit < 0 && past_at(c)) hit = v0 + j;
                    }
                }
                const unsigned hits = __ballot_sync(0xffffffffu, hit >= 0), poss = __ballot_sync(0xffffffffu, pos >= 0);
                const int from = hits ? __ffs(hits) - 1 : 31 - __clz(poss | 1u);
                const int tok = __shfl_sync(0xffffffffu, hits ? hit : pos, from);
                if (lane == 0) a.next_token[b] = tok;
            }
            break;
        }
        // the same decision in every CTA of the cluster: all go on to the second pass together
        if (pass == 1 && rank == 0 && threadIdx.x == 0) a.next_token[b] = -1;
        row.q = nullptr;
        row.certain = -1;
        __syncthreads();
    }
    cluster.sync();  // no CTA leaves while another still reads its total
}

}  // namespace

cudaError_t launch_verify_accept(const AcceptArgs &a, cudaStream_t stream) {
    // One CTA per 8192 weights, at most eight: a row of 65536 then has 8 x 256 threads with 16
    // loads each in flight, and a short row pays for no cluster.  But a CTA that only starts when
    // another ends adds that one's start and end (about 10 us of loads that depend on one another) to
    // its own: while there are more than fit the SMs at once, fewer and longer ones.  256 rows of
    // 100003: 59 us in clusters of eight, 49 of four, 47 of two, 52 of one.
    constexpr int kResident = 152 * kCtasPerSm, kMostSegs = 8192;
    const int segs = (a.V + kSeg - 1) / kSeg;
    int ranks = 1;
    while (ranks < 8 && static_cast<long long>(ranks) * 8192 < a.V) ranks *= 2;
    while (ranks > 1 && static_cast<long long>(a.B) * ranks > kResident && (segs + ranks / 2 - 1) / (ranks / 2) <= kMostSegs) ranks /= 2;
    const int per = (segs + ranks - 1) / ranks;
    const int smem = per * static_cast<int>(sizeof(Pair));  // at most 64 KB
    if (smem > 40 * 1024) {
        static std::atomic<unsigned long long> allowed{0};
        const cudaError_t e = gdr_allow_smem(reinterpret_cast<const void *>(wkv7_verify_accept_kernel),
                                             kMostSegs * static_cast<int>(sizeof(Pair)), allowed);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ranks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.stream = stream;
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ranks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    return cudaLaunchKernelEx(&cfg, wkv7_verify_accept_kernel, a, per);
}

}  // namespace wkv7
