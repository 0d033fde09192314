// gdn_norm.cu -- the norms around a mixer, each fused with what stands next to it.
//
// gated_norm: the output norm of each head with its gate,
//     y = x / sqrt(mean_i x_i^2 + eps) * w * act(z)         (norm, then gate)
//     y = u / sqrt(mean_i u_i^2 + eps) * w,  u = x act(z)   (GDN_GATE_FIRST)
// residual_norm: from one block to the next,
//     u  = y / sqrt(mean y^2 + eps) * w_post   (y itself without w_post)
//     x' = x + s act(g) u
//     h  = x' / sqrt(mean x'^2 + eps) * w_pre
//
// Both are bound by HBM: every input element is read once, kept in registers
// in fp32 across the reductions, and every output element written once.  A
// row is spread over a group of threads (part of a warp, or a whole CTA), each
// holding ITEMS 16-byte vectors of it.  Sums of squares are fp32; h is formed
// from the unrounded x'.
#include <atomic>

#include "gdn_internal.cuh"

namespace gdn {
namespace {

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T v[VEC];
};

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T *p, float (&x)[VEC]) {
    if constexpr (sizeof(T) * VEC > 16) {  // fp32 beside a 16-bit vector: two 16-byte loads
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(p + j);
            x[j] = f.x; x[j + 1] = f.y; x[j + 2] = f.z; x[j + 3] = f.w;
        }
    } else {
        const Pack<T, VEC> u = *reinterpret_cast<const Pack<T, VEC> *>(p);
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = ld_f(&u.v[j]);
    }
}
// VEC elements as they are stored, loaded ahead of their use.
template <typename T, int VEC>
struct Raw {
    static constexpr int kPacks = sizeof(T) * VEC > 16 ? (int)(sizeof(T) * VEC / 16) : 1;
    Pack<T, VEC / kPacks> v[kPacks];
    __device__ __forceinline__ void load(const T *p) {
#pragma unroll
        for (int k = 0; k < kPacks; ++k) v[k] = reinterpret_cast<const Pack<T, VEC / kPacks> *>(p)[k];
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < kPacks; ++k)
#pragma unroll
            for (int j = 0; j < VEC / kPacks; ++j) v[k].v[j] = T(0.f);
    }
    __device__ __forceinline__ void get(float (&x)[VEC]) const {
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = at(j);
    }
    __device__ __forceinline__ float at(int j) const { return ld_f(&v[j / (VEC / kPacks)].v[j % (VEC / kPacks)]); }
};
__device__ __forceinline__ void st_pair(float *p, float a, float b) { *reinterpret_cast<float2 *>(p) = make_float2(a, b); }
__device__ __forceinline__ void st_pair(__half *p, float a, float b) {
    *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(a, b);
}
__device__ __forceinline__ void st_pair(__nv_bfloat16 *p, float a, float b) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        st_out(p, x[0]);
    } else {
        constexpr int P = 16 / (int)sizeof(T);  // elements of a 16-byte store
#pragma unroll
        for (int j = 0; j < VEC; j += P) {
            Pack<T, P> u;
#pragma unroll
            for (int e = 0; e < P; e += 2) st_pair(&u.v[e], x[j + e], x[j + e + 1]);
            *reinterpret_cast<Pack<T, P> *>(p + j) = u;
        }
    }
}

// VEC weights from element i on, of runtime type (vectors: 16-byte aligned);
// ones without weights.
template <int VEC>
__device__ __forceinline__ void load_weight(const void *w, int i, int dt, float offset, float (&x)[VEC]) {
    if (w == nullptr) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = 1.f;
        return;
    }
    if (dt == GDN_F32) load_vec<float, VEC>(reinterpret_cast<const float *>(w) + i, x);
    else if (dt == GDN_F16) load_vec<__half, VEC>(reinterpret_cast<const __half *>(w) + i, x);
    else load_vec<__nv_bfloat16, VEC>(reinterpret_cast<const __nv_bfloat16 *>(w) + i, x);
    if (offset != 0.f)
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] += offset;
}

// 1 / (1 + e^-z) by the base-2 exponential and the reciprocal of the PTX ISA
// (relative errors 2^-22 and 2^-23), in place.  For 16-bit values the rounding of
// z log2 e is as far below their own as those; fp32 takes its rest along.
template <typename T, int VEC>
__device__ __forceinline__ void sigmoid_of(float (&z)[VEC]) {
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        const float t = -1.4426950408889634f * z[j];
        float e, s;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
        if constexpr (sizeof(T) == 4) {
            const float rest = fmaf(-1.4426950408889634f, z[j], -t);
            const float more = e * (0.6931471805599453f * rest);
            e = t < 126.f ? e + more : e;  // (no rest beside an infinite e)
        }
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
        z[j] = s;
    }
}
// act(z), in place; the branches are the same for every thread.
template <typename T, int VEC>
__device__ __forceinline__ void activate(float (&z)[VEC], int act) {
    float s[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[j] = z[j];
    sigmoid_of<T, VEC>(s);
    if (act == GDN_GATE_SILU) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) z[j] *= s[j];
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) z[j] = s[j];
    }
}

// Sum over the row's group of threads: `lanes` (a power of two) threads of a
// warp, or, with lanes > 32, all threads of the CTA.  red: a float for each
// warp, another buffer in every second call.
__device__ __forceinline__ float row_sum(float x, int lanes, float *red) {
    for (int o = (lanes < 32 ? lanes : 32) / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lanes <= 32) return x;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) red[warp] = x;
    __syncthreads();
    float s = lane < nw ? red[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Rows on their way.  With vectors, each thread copies its own 16-byte pieces of
// its next rows to shared memory, `depth` rows deep (cp.async: no other thread
// reads them, so no barrier stands between copy and use); without, the next row
// waits in registers.  NP: pieces of a row a thread.
template <int NP>
struct Ring {
    uint4 *mine;
    __device__ __forceinline__ Ring(uint4 *base) : mine(base + threadIdx.x) {}
    __device__ __forceinline__ uint4 *at(int slot, int piece) const { return mine + (slot * NP + piece) * blockDim.x; }
    __device__ __forceinline__ void copy(int slot, int piece, const void *src) const {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         static_cast<uint32_t>(__cvta_generic_to_shared(at(slot, piece)))),
                     "l"(src)
                     : "memory");
    }
    __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // all but the last `depth` - 1 rows copied
    __device__ __forceinline__ static void wait(int depth) {
        if (depth == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
        else if (depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
        else if (depth == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    template <typename R>
    __device__ __forceinline__ void get(int slot, int piece, R &raw) const {
#pragma unroll
        for (int k = 0; k < R::kPacks; ++k) *reinterpret_cast<uint4 *>(&raw.v[k]) = *at(slot, piece + k);
    }
    __device__ __forceinline__ void clear(int depth) const {
        for (int s = 0; s < depth; ++s)
            for (int k = 0; k < NP; ++k) *at(s, k) = make_uint4(0u, 0u, 0u, 0u);
    }
};
constexpr int kRingBytes = 98304;  // most of a CTA's ring: two CTAs an SM
__host__ __device__ constexpr int ring_depth(int np, int threads) {
    const int d = kRingBytes / (np * threads * 16);
    return d > 4 ? 4 : d < 1 ? 1 : d;
}

constexpr int kThreads = 256;
// Largest CTA that spread() asks for: only scalar rows beyond 8192 elements take more than 512 threads.
template <int VEC>
constexpr int kMaxThreads = VEC > 1 ? 512 : 1024;

template <typename T, int VEC, int ITEMS>
__global__ void __launch_bounds__(kMaxThreads<VEC>) gated_norm_kernel(const GatedNormParams p, int lanes) {
    __shared__ float red[2][32];
    const int per_cta = blockDim.x / lanes;
    const unsigned rows = (unsigned)(p.N * p.H), H = (unsigned)p.H;
    const int t = threadIdx.x % lanes;
    const int act = p.gate & 0xF;
    const bool first = (p.gate & GDN_GATE_FIRST) != 0;
    const float offset = (p.gate & GDN_NORM_UNIT_OFFSET) ? 1.f : 0.f;
    const float inv_d = 1.f / (float)p.d;
    // the thread's columns, and so its weights, are the same in every row
    float w[ITEMS][VEC];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = (k * lanes + t) * VEC;
        if (i < p.d) load_weight<VEC>(p.w, i, p.dt_w, offset, w[k]);
    }
    constexpr int NP = 2 * ITEMS;
    extern __shared__ uint4 ring_smem[];
    const Ring<NP> ring(ring_smem);
    const int depth = VEC > 1 ? ring_depth(NP, blockDim.x) : 1;
    Raw<T, VEC> nx[ITEMS], nz[ITEMS];
    auto fetch = [&](unsigned r, int slot) {
        const unsigned n = r / H, h = r - n * H;
        const T *x = reinterpret_cast<const T *>(p.x) + (int64_t)n * p.xs + (int64_t)h * p.d;
        const T *z = reinterpret_cast<const T *>(p.z) + (int64_t)n * p.zs + (int64_t)h * p.d;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = (k * lanes + t) * VEC;
            if (i < p.d) {
                if constexpr (VEC > 1) {
                    ring.copy(slot, 2 * k, x + i);
                    if (act != GDN_GATE_NONE) ring.copy(slot, 2 * k + 1, z + i);
                } else {
                    nx[k].load(x + i);
                    if (act != GDN_GATE_NONE) nz[k].load(z + i);
                }
            }
        }
    };
    // (every thread of a CTA takes as many turns: the sums are taken together)
    const unsigned r0 = blockIdx.x * per_cta, step = gridDim.x * per_cta, mine = threadIdx.x / lanes;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) nx[k].clear(), nz[k].clear();
    if constexpr (VEC > 1) {
        ring.clear(depth);
        for (int k = 0; k < depth - 1; ++k) {
            if (r0 + mine + k * step < rows) fetch(r0 + mine + k * step, k);
            ring.commit();
        }
    } else if (r0 + mine < rows) {
        fetch(r0 + mine, 0);
    }
    int turn = 0, slot = 0;
    for (unsigned base = r0; base < rows; base += step, ++turn) {
        const unsigned r = base + mine;
        const bool live = r < rows;
        if constexpr (VEC > 1) {
            const unsigned ahead = (depth - 1) * step;
            if (r + ahead < rows) fetch(r + ahead, slot == 0 ? depth - 1 : slot - 1);
            ring.commit();
            ring.wait(depth);
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                ring.get(slot, 2 * k, nx[k]);
                if (act != GDN_GATE_NONE) ring.get(slot, 2 * k + 1, nz[k]);
            }
            slot = slot + 1 == depth ? 0 : slot + 1;
        }
        float a[ITEMS][VEC], g[ITEMS][VEC];
        float ss = 0.f;
        // (columns past the row and rows past the last hold zeros or old values)
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            nx[k].get(a[k]);
            if (act != GDN_GATE_NONE) {
                nz[k].get(g[k]);
                activate<T, VEC>(g[k], act);
                if (first)
#pragma unroll
                    for (int j = 0; j < VEC; ++j) a[k][j] *= g[k][j];
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) ss = fmaf(a[k][j], a[k][j], ss);
        }
        if constexpr (VEC == 1)
            if (r + step < rows) fetch(r + step, 0);
        ss = row_sum(ss, lanes, red[turn & 1]);
        const float rs = rsqrtf(fmaf(ss, inv_d, p.eps));
        if (live) {
            const unsigned n = r / H, h = r - n * H;
            T *y = reinterpret_cast<T *>(p.out) + (int64_t)n * p.os + (int64_t)h * p.d;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int i = (k * lanes + t) * VEC;
                if (i < p.d) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) a[k][j] *= rs * w[k][j];
                    if (act != GDN_GATE_NONE && !first)
#pragma unroll
                        for (int j = 0; j < VEC; ++j) a[k][j] *= g[k][j];
                    store_vec<T, VEC>(y + i, a[k]);
                }
            }
        }
    }
}

template <typename T, typename TR, int VEC, int ITEMS>
__global__ void __launch_bounds__(kMaxThreads<VEC>) residual_norm_kernel(const ResidualNormParams p, int lanes) {
    __shared__ float red[2][32];
    const int per_cta = blockDim.x / lanes, t = threadIdx.x % lanes;
    const int act = p.flags & 0xF;
    const float offset = (p.flags & GDN_NORM_UNIT_OFFSET) ? 1.f : 0.f;
    const float inv_d = 1.f / (float)p.D;
    constexpr int XP = Raw<TR, VEC>::kPacks, NP = (2 + XP) * ITEMS;
    extern __shared__ uint4 ring_smem[];
    const Ring<NP> ring(ring_smem);
    const int depth = VEC > 1 ? ring_depth(NP, blockDim.x) : 1;
    Raw<T, VEC> ny[ITEMS], nz[ITEMS];
    Raw<TR, VEC> nx[ITEMS];
    auto fetch = [&](int64_t n, int slot) {
        const T *y = reinterpret_cast<const T *>(p.y) + n * p.ys;
        const T *z = reinterpret_cast<const T *>(p.z) + n * p.zs;
        const TR *x = reinterpret_cast<const TR *>(p.x) + n * p.D;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = (k * lanes + t) * VEC;
            if (i < p.D) {
                if constexpr (VEC > 1) {
                    ring.copy(slot, (2 + XP) * k, y + i);
                    if (act != GDN_GATE_NONE) ring.copy(slot, (2 + XP) * k + 1, z + i);
                    if (p.x != nullptr)
#pragma unroll
                        for (int e = 0; e < XP; ++e) ring.copy(slot, (2 + XP) * k + 2 + e, x + i + e * (VEC / XP));
                } else {
                    ny[k].load(y + i);
                    if (act != GDN_GATE_NONE) nz[k].load(z + i);
                    if (p.x != nullptr) nx[k].load(x + i);
                }
            }
        }
    };
    // (every thread of a CTA takes as many turns: the sums are taken together)
    const int64_t step = (int64_t)gridDim.x * per_cta, mine = threadIdx.x / lanes;
    int64_t base = (int64_t)blockIdx.x * per_cta;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) ny[k].clear(), nz[k].clear(), nx[k].clear();
    if constexpr (VEC > 1) {
        ring.clear(depth);
        for (int k = 0; k < depth - 1; ++k) {
            if (base + mine + k * step < p.N) fetch(base + mine + k * step, k);
            ring.commit();
        }
    } else if (base + mine < p.N) {
        fetch(base + mine, 0);
    }
    int slot = 0;
    for (; base < p.N; base += step) {
        const int64_t n = base + mine;
        const bool live = n < p.N;
        if constexpr (VEC > 1) {
            const int64_t ahead = (depth - 1) * step;
            if (n + ahead < p.N) fetch(n + ahead, slot == 0 ? depth - 1 : slot - 1);
            ring.commit();
            ring.wait(depth);
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                ring.get(slot, (2 + XP) * k, ny[k]);
                if (act != GDN_GATE_NONE) ring.get(slot, (2 + XP) * k + 1, nz[k]);
                if (p.x != nullptr) ring.get(slot, (2 + XP) * k + 2, nx[k]);
            }
            slot = slot + 1 == depth ? 0 : slot + 1;
        }
        float u[ITEMS][VEC], a[ITEMS][VEC], ss = 0.f;
        // (columns past the row and rows past the last hold zeros or old values)
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            ny[k].get(u[k]);
            nx[k].get(a[k]);
            if (p.w_post != nullptr)
#pragma unroll
                for (int j = 0; j < VEC; ++j) ss = fmaf(u[k][j], u[k][j], ss);
            if (act != GDN_GATE_NONE) {
                float g[VEC];
                nz[k].get(g);
                activate<T, VEC>(g, act);
#pragma unroll
                for (int j = 0; j < VEC; ++j) u[k][j] *= g[j];
            }
        }
        if constexpr (VEC == 1)
            if (n + step < p.N) fetch(n + step, 0);
        float rs = p.scale;
        if (p.w_post != nullptr) rs *= rsqrtf(fmaf(row_sum(ss, lanes, red[0]), inv_d, p.eps));
        ss = 0.f;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = (k * lanes + t) * VEC;
            if (live && i < p.D) {
                if (p.w_post != nullptr) {
                    float w[VEC];
                    load_weight<VEC>(p.w_post, i, p.dt_w, offset, w);
#pragma unroll
                    for (int j = 0; j < VEC; ++j) u[k][j] *= w[j];
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    a[k][j] = fmaf(rs, u[k][j], a[k][j]);
                    ss = fmaf(a[k][j], a[k][j], ss);
                }
                if (p.x_out != nullptr) store_vec<TR, VEC>(reinterpret_cast<TR *>(p.x_out) + n * p.D + i, a[k]);
            }
        }
        if (p.out == nullptr) {
            if (lanes > 32) __syncthreads();  // the next turn writes red[0] again
            continue;
        }
        rs = rsqrtf(fmaf(row_sum(ss, lanes, red[1]), inv_d, p.eps));
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = (k * lanes + t) * VEC;
            if (live && i < p.D) {
                float w[VEC];
                load_weight<VEC>(p.w_pre, i, p.dt_w, offset, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) a[k][j] *= rs * w[j];
                store_vec<T, VEC>(reinterpret_cast<T *>(p.out) + n * p.D + i, a[k]);
            }
        }
        // without the first sum no barrier stands between this one and the next turn's
        if (p.w_post == nullptr && lanes > 32) __syncthreads();
    }
}

// How a row of `width` elements is spread: `lanes` threads of ITEMS vectors
// each, `threads` a CTA.  Rows of up to 32 vectors take the smallest power of
// two of lanes of one vector each, so several rows share a warp; longer rows
// take a warp of up to four vectors a lane, then a whole CTA.
struct Spread {
    int lanes, threads, items;
};
Spread spread(int width, int vec) {
    const int nv = (width + vec - 1) / vec;
    if (nv <= 128) {
        int lanes = 1;
        while (lanes < 32 && lanes < nv) lanes *= 2;
        int items = 1;
        while (lanes * items < nv) items *= 2;
        return {lanes, kThreads, items};
    }
    int items = 1;
    while ((nv + items - 1) / items > 512 && items < 16) items *= 2;
    const int threads = ((nv + items - 1) / items + 31) / 32 * 32;
    // one warp is a group of its own; more are a CTA
    return {threads, threads, items};
}

template <int N>
struct Int {
    static constexpr int value = N;
};
template <typename F>
cudaError_t with_items(int items, F f) {
    switch (items) {
        case 1: return f(Int<1>{});
        case 2: return f(Int<2>{});
        case 4: return f(Int<4>{});
        case 8: return f(Int<8>{});
        default: return f(Int<16>{});
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// CTAs of `threads` threads that run at once, asked once for each kernel and size
// (0: the question failed).  NP: the pieces of its ring, 0 without one.
template <auto Kern, int NP>
unsigned resident(int threads, int bytes) {
    static std::atomic<int> cache[33];
    int c = cache[threads / 32].load(std::memory_order_relaxed);
    if (c == 0) {
        if (NP > 0 && set_smem_once<Kern>(2 * kRingBytes) != cudaSuccess) return 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&c, Kern, threads, bytes) != cudaSuccess || c < 1) return 0;
        cache[threads / 32].store(c, std::memory_order_relaxed);
    }
    return (unsigned)(c * sm_count_of_current_device());
}
template <auto Kern, int NP, typename P>
cudaError_t launch_rows(const P &p, const Spread &s, int64_t rows, cudaStream_t stream) {
    const int64_t per = s.threads / s.lanes, ctas = (rows + per - 1) / per;
    const int bytes = NP > 0 ? ring_depth(NP, s.threads) * NP * s.threads * 16 : 0;
    const unsigned most = resident<Kern, NP>(s.threads, bytes);
    if (most == 0) return cudaErrorInvalidConfiguration;
    Kern<<<ctas < most ? (unsigned)ctas : most, s.threads, bytes, stream>>>(p, s.lanes);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_gated_t(const GatedNormParams &p, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    // 16-byte vectors where every row of x, z and out starts on 16 bytes
    const bool vec = p.d % V == 0 && p.xs % V == 0 && p.os % V == 0 && (p.z == nullptr || p.zs % V == 0) &&
                     aligned16(p.x) && aligned16(p.z) && aligned16(p.out) && aligned16(p.w);
    const Spread s = spread(p.d, vec ? V : 1);
    return with_items(s.items, [&](auto items) {
        constexpr int I = decltype(items)::value;
        constexpr int IV = I > 32 / V ? 32 / V : I;  // (a row has 32 elements a thread at most)
        return vec ? launch_rows<gated_norm_kernel<T, V, IV>, 2 * IV>(p, s, p.N * p.H, stream)
                   : launch_rows<gated_norm_kernel<T, 1, I>, 0>(p, s, p.N * p.H, stream);
    });
}

template <typename T, typename TR>
cudaError_t launch_residual_t(const ResidualNormParams &p, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool vec = p.D % V == 0 && p.ys % V == 0 && (p.z == nullptr || p.zs % V == 0) && aligned16(p.y) &&
                     aligned16(p.z) && aligned16(p.x) && aligned16(p.x_out) && aligned16(p.out) &&
                     aligned16(p.w_post) && aligned16(p.w_pre);
    const Spread s = spread(p.D, vec ? V : 1);
    return with_items(s.items, [&](auto items) {
        constexpr int I = decltype(items)::value;
        constexpr int IV = I > 32 / V ? 32 / V : I;  // (a row has 32 elements a thread at most)
        constexpr int NP = (2 + (sizeof(TR) > sizeof(T) ? 2 : 1)) * IV;
        return vec ? launch_rows<residual_norm_kernel<T, TR, V, IV>, NP>(p, s, p.N, stream)
                   : launch_rows<residual_norm_kernel<T, TR, 1, I>, 0>(p, s, p.N, stream);
    });
}

}  // namespace

cudaError_t launch_gated_norm(const GatedNormParams &p, cudaStream_t stream) {
    switch (p.dt_x) {
        case GDN_F32: return launch_gated_t<float>(p, stream);
        case GDN_F16: return launch_gated_t<__half>(p, stream);
        default: return launch_gated_t<__nv_bfloat16>(p, stream);
    }
}

cudaError_t launch_residual_norm(const ResidualNormParams &p, cudaStream_t stream) {
    const bool wide = p.dt_res == GDN_F32;
    switch (p.dt_x) {
        case GDN_F32: return launch_residual_t<float, float>(p, stream);
        case GDN_F16:
            return wide ? launch_residual_t<__half, float>(p, stream) : launch_residual_t<__half, __half>(p, stream);
        default:
            return wide ? launch_residual_t<__nv_bfloat16, float>(p, stream)
                        : launch_residual_t<__nv_bfloat16, __nv_bfloat16>(p, stream);
    }
}

}  // namespace gdn
