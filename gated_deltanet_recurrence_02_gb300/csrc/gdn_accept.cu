// gdn_accept.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers (speculative sampling).
//
// Row b has c_b drafts x_0 .. x_{c-1}, the target's distributions p_0 .. p_K
// and the drafts' q_0 .. q_{K-1} (without them q_i(x_i) = 1: a lookup's or a
// greedy draft's certainty):
//   n      = the first i < c with u_i q_i(x_i) >= p_i(x_i), else c
//   weight = max(p_n - q_n, 0) if n < c, else p_c;  p_n where that is 0 everywhere
//   token  = the first j with weight_0 + .. + weight_j > goal
// The weights are taken in whole units of 2^-40, so that their sums are exact
// 64-bit integers and do not depend on the order or the split of the work:
// goal = floor(u_K * total) is the same for every launch shape.  The token has a
// random number of its own: given a rejection, the tests' ones are no longer
// uniform.
//
// Of B (2K + 1) rows of V probabilities only two rows a request are read, by a cluster
// of CTAs: each warp sums a contiguous segment, the warps' sums are shared through
// distributed shared memory, and the CTA that owns the segment with the goal scans it
// again (from L2) for the token.  For many requests bound by HBM and by what surrounds
// the one read of the rows, a chain of dependent accesses: the drafts, their
// probabilities, the rows, the cluster's sums, the segment.  128 requests of 100003 fp32
// probabilities, 4 drafts: 25 us (15 us of HBM time, 0.6 of the copy bandwidth; 47 us with
// conversions to 64-bit integers); 1 request of 32000 bf16 ones without draft
// probabilities: 8.3 us, the chain.
#include <cooperative_groups.h>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxCluster = 8;
constexpr int kCtas = 8;  // on a multiprocessor at once, which leaves 32 registers a thread (28 bytes spill)

// Weights in whole units of 2^-40, floor(w 2^40) for w clamped to [0, 1] (NaN: 0).
// A conversion to a 64-bit integer runs at a fraction of the load rate, so the two
// halves of 20 bits are read off sums with 2^23 that are rounded down: floor(w 2^20)
// are the low bits of the first, the rest of w goes into the second exactly, and
// each half is summed in 32 bits over a few weights before it joins the total.
struct Units {
    uint32_t hi = 0, lo = 0;
    __device__ __forceinline__ void add(float w) {
        w = __saturatef(w);
        const float a = __fmaf_rz(w, 1048576.f, 8388608.f);
        const float rest = fmaf(w, 1048576.f, 8388608.f - a);
        const float b = __fmaf_rz(rest, 1048576.f, 8388608.f);
        hi += __float_as_uint(a) - 0x4B000000u;
        lo += __float_as_uint(b) - 0x4B000000u;
    }
    __device__ __forceinline__ long long total() const { return ((long long)hi << 20) + lo; }
};
__device__ __forceinline__ long long units(float w) {
    Units u;
    u.add(w);
    return u.total();
}

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

template <typename T>
struct Row {
    const T *p, *q;   // q: nullptr if nothing is taken off
    int drop;         // token whose weight is 0 (the rejected one of a certain draft), or -1
    __device__ __forceinline__ float weight(int j) const {
        const float t = ld_f(p + j);
        return q != nullptr ? t - ld_f(q + j) : t;
    }
    __device__ __forceinline__ long long at(int j) const { return j == drop ? 0ll : units(weight(j)); }
};

// Sum over tokens lo .. hi - 1 by a warp, VEC tokens a load.  hi - lo need not be a
// multiple; with VEC > 1 lo is one, and rows are aligned to VEC tokens.
template <typename T, int VEC, bool Q>
__device__ __forceinline__ long long segment_sum(const Row<T> &row, int lo, int hi, int lane) {
    constexpr int N = (VEC > 1 ? 4 : 8) / (Q ? 2 : 1);  // loads of a row in flight
    long long s = 0;
    int j = lo + lane * VEC;
    for (; j + ((N - 1) * 32 + 1) * VEC <= hi; j += N * 32 * VEC) {
        Pack<T, VEC> a[N], b[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            a[i] = *reinterpret_cast<const Pack<T, VEC> *>(row.p + j + i * 32 * VEC);
            if constexpr (Q) b[i] = *reinterpret_cast<const Pack<T, VEC> *>(row.q + j + i * 32 * VEC);
        }
        Units u;
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < VEC; ++e) u.add(Q ? ld_f(&a[i].v[e]) - ld_f(&b[i].v[e]) : ld_f(&a[i].v[e]));
        s += u.total();
    }
    for (; j < hi; j += 32 * VEC)
        for (int e = 0; e < VEC && j + e < hi; ++e) s += units(row.weight(j + e));
    if (lo <= row.drop && row.drop < hi && lane == 0) s -= units(row.weight(row.drop));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, kCtas) accept_kernel(const AcceptParams p) {
    __shared__ long long seg[kWarps];                 // this CTA's segment sums, read by the cluster
    __shared__ long long all[kMaxCluster * kWarps];   // the cluster's, in token order
    __shared__ long long part[kWarps];
    __shared__ int n_sh;
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = (int)cluster.block_rank(), cs = (int)cluster.num_blocks();
    const int b = blockIdx.x / cs;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int K = p.K, V = p.V;
    const T *P = reinterpret_cast<const T *>(p.p), *Q = reinterpret_cast<const T *>(p.q);
    const int32_t *x = p.drafts + (long)b * K;
    const float *u = p.u + (long)b * (K + 1);
    int c = K;
    if (p.count != nullptr) c = min(max(p.count[b], 0), K);

    if (warp == 0) {
        int n = c;
        for (int i0 = 0; i0 < c; i0 += 32) {
            const int i = i0 + lane;
            bool ok = true;
            if (i < c) {
                const int tok = x[i];
                ok = false;
                if (tok >= 0 && tok < V) {
                    const float pt = ld_f(P + ((int64_t)b * (K + 1) + i) * p.ps + tok);
                    const float qt = Q != nullptr ? ld_f(Q + ((int64_t)b * K + i) * p.qs + tok) : 1.f;
                    ok = u[i] * qt < pt;
                } else if (rank == 0) {
                    atomicOr(p.err, (uint32_t)GDN_DEVERR_BAD_INDEX);
                }
            }
            const unsigned bad = __ballot_sync(0xffffffffu, !ok);
            if (bad != 0) {
                n = i0 + __ffs(bad) - 1;
                break;
            }
        }
        if (lane == 0) n_sh = n;
    }
    __syncthreads();
    const int n = n_sh;
    Row<T> row;
    row.p = P + ((int64_t)b * (K + 1) + n) * p.ps;
    row.q = (n < c && Q != nullptr) ? Q + ((int64_t)b * K + n) * p.qs : nullptr;
    row.drop = (n < c && Q == nullptr) ? x[n] : -1;
    const int nseg = cs * kWarps;
    const int len = ((V + nseg - 1) / nseg + VEC - 1) / VEC * VEC;
    const int mine = rank * kWarps + warp;
    const int lo = (int)min((int64_t)mine * len, (int64_t)V), hi = min(lo + len, V);

    long long total = 0;
    for (int pass = 0; pass < 2; ++pass) {
        const long long s = row.q != nullptr ? segment_sum<T, VEC, true>(row, lo, hi, lane)
                                             : segment_sum<T, VEC, false>(row, lo, hi, lane);
        if (lane == 0) seg[warp] = s;
        cluster.sync();
        for (int i = threadIdx.x; i < nseg; i += kThreads) all[i] = cluster.map_shared_rank(seg, i / kWarps)[i % kWarps];
        cluster.sync();  // every CTA has its copy: seg may be written again, or its CTA end
        total = 0;
        for (int i = lane; i < nseg; i += 32) total += all[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        if (total > 0 || (row.q == nullptr && row.drop < 0)) break;
        // nothing is left of the target: it is sampled as it is
        row.q = nullptr;
        row.drop = -1;
    }

    int32_t *out = p.tokens + (long)b * (K + 1);
    if (rank == 0) {
        for (int i = threadIdx.x; i <= K; i += kThreads)
            if (i != n || total == 0) out[i] = i < n ? x[i] : -1;
        if (threadIdx.x == 0) p.emitted[b] = n + 1;
    }
    if (total == 0) return;
    long long goal = (long long)((double)u[K] * (double)total);
    goal = goal < 0 ? 0 : (goal >= total ? total - 1 : goal);
    // the segment whose running sum first exceeds the goal
    long long before = 0;
    int hit = 0;
    for (int i0 = 0; i0 < nseg; i0 += 32) {
        long long v = i0 + lane < nseg ? all[i0 + lane] : 0;
        const long long own = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += t;
        }
        const unsigned over = __ballot_sync(0xffffffffu, before + v > goal);
        if (over != 0) {
            const int l = __ffs(over) - 1;
            hit = i0 + l;
            before += __shfl_sync(0xffffffffu, v - own, l);
            break;
        }
        before += __shfl_sync(0xffffffffu, v, 31);
    }
    if (hit / kWarps != rank) return;
    // its tokens, a run of consecutive ones for each thread
    const int s_lo = (int)min((int64_t)hit * len, (int64_t)V), s_hi = min(s_lo + len, V);
    const int per = (len + kThreads - 1) / kThreads;
    const int t_lo = min(s_lo + (int)threadIdx.x * per, s_hi), t_hi = min(t_lo + per, s_hi);
    long long s = 0;
    for (int j = t_lo; j < t_hi; ++j) s += row.at(j);
    long long incl = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
    }
    if (lane == 31) part[warp] = incl;
    __syncthreads();
    long long run = before + incl - s;
    for (int w = 0; w < warp; ++w) run += part[w];
    if (run <= goal && run + s > goal) {  // one thread: the running sum crosses the goal in its run
        for (int j = t_lo; j < t_hi; ++j) {
            run += row.at(j);
            if (run > goal) {
                out[n] = j;
                break;
            }
        }
    }
}

template <typename T>
cudaError_t launch_t(const AcceptParams &p, cudaStream_t stream) {
    // CTAs a row: more while all of them run at once and each warp still sums a few
    // hundred tokens (128 requests of 100003 fp32 tokens: 25 us as 1024 CTAs of 256 threads;
    // 34 with room for six of them on a multiprocessor, a second wave; 37 as 512 CTAs of
    // 512 threads, of which some multiprocessors had one more than others)
    int cs = 1;
    const long slots = (long)kCtas * sm_count_of_current_device();
    while (cs < kMaxCluster && (long)p.B * cs * 2 <= slots && p.V / (2 * cs * kWarps) >= 128) cs *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(p.B * cs));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)cs;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    constexpr int W = 16 / (int)sizeof(T);
    const bool vec = p.ps % W == 0 && (p.q == nullptr || p.qs % W == 0) &&
                     ((reinterpret_cast<uintptr_t>(p.p) | reinterpret_cast<uintptr_t>(p.q)) & 15) == 0;
    const cudaError_t e = vec ? cudaLaunchKernelEx(&cfg, accept_kernel<T, W>, p)
                              : cudaLaunchKernelEx(&cfg, accept_kernel<T, 1>, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_accept(const AcceptParams &p, cudaStream_t stream) {
    switch (p.dt) {
        case GDN_F32: return launch_t<float>(p, stream);
        case GDN_F16: return launch_t<__half>(p, stream);
        default: return launch_t<__nv_bfloat16>(p, stream);
    }
}

}  // namespace gdn
