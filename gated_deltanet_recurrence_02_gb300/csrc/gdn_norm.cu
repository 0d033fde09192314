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
template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T *p, const float (&x)[VEC]) {
    if constexpr (sizeof(T) * VEC > 16) {
#pragma unroll
        for (int j = 0; j < VEC; j += 4)
            *reinterpret_cast<float4 *>(p + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
    } else {
        Pack<T, VEC> u;
#pragma unroll
        for (int j = 0; j < VEC; ++j) st_out(&u.v[j], x[j]);
        *reinterpret_cast<Pack<T, VEC> *>(p) = u;
    }
}

// VEC weights from element i on, of runtime type; ones without weights.
template <int VEC>
__device__ __forceinline__ void load_weight(const void *w, int i, int dt, float offset, float (&x)[VEC]) {
    if (w == nullptr) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = 1.f;
        return;
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = ld_gate(w, i + j, dt) + offset;
}

// silu(z) or sigmoid(z).  With 16-bit storage the fast exponential and divide
// are far below the rounding of the result.
template <typename T>
__device__ __forceinline__ float activation(float z, int act) {
    float s;
    if constexpr (sizeof(T) == 2) s = __fdividef(1.f, 1.f + __expf(-z));
    else s = 1.f / (1.f + expf(-z));
    return act == GDN_GATE_SILU ? z * s : s;
}

// Sum over the row's group of threads: `lanes` (a power of two) threads of a
// warp, or, with lanes > 32, all threads of the CTA (red: one float a warp and
// the total; safe to call again after the next __syncthreads-ordered call).
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

constexpr int kThreads = 256;
// Largest CTA that spread() asks for: only scalar rows beyond 8192 elements take more than 512 threads.
template <int VEC>
constexpr int kMaxThreads = VEC > 1 ? 512 : 1024;

template <typename T, int VEC, int ITEMS>
__global__ void __launch_bounds__(kMaxThreads<VEC>) gated_norm_kernel(const GatedNormParams p, int lanes) {
    __shared__ float red[32];
    const int per_cta = blockDim.x / lanes;
    const int64_t rows = p.N * p.H;
    const int64_t r = (int64_t)blockIdx.x * per_cta + threadIdx.x / lanes;
    const int t = threadIdx.x % lanes;
    const bool live = r < rows;  // a dead row's threads still take part in the shuffles
    const int64_t n = live ? r / p.H : 0;
    const int h = (int)(live ? r - n * p.H : 0);
    const T *x = reinterpret_cast<const T *>(p.x) + n * p.xs + (int64_t)h * p.d;
    const T *z = reinterpret_cast<const T *>(p.z) + n * p.zs + (int64_t)h * p.d;
    T *y = reinterpret_cast<T *>(p.out) + n * p.os + (int64_t)h * p.d;
    const int act = p.gate & 0xF;
    const bool first = (p.gate & GDN_GATE_FIRST) != 0;
    const float offset = (p.gate & GDN_NORM_UNIT_OFFSET) ? 1.f : 0.f;
    float a[ITEMS][VEC], g[ITEMS][VEC];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = (k * lanes + t) * VEC;
        const bool in = live && i < p.d;
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[k][j] = 0.f, g[k][j] = 0.f;
        if (in) load_vec<T, VEC>(x + i, a[k]);
        if (in && act != GDN_GATE_NONE) load_vec<T, VEC>(z + i, g[k]);
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            g[k][j] = act != GDN_GATE_NONE ? activation<T>(g[k][j], act) : 1.f;
            if (first) a[k][j] *= g[k][j];
            // elements past the row are zeros, and stay zeros through a gate
            ss = fmaf(a[k][j], a[k][j], ss);
        }
    ss = row_sum(ss, lanes, red);
    const float rs = 1.f / sqrtf(ss / (float)p.d + p.eps);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = (k * lanes + t) * VEC;
        if (live && i < p.d) {
            float w[VEC];
            load_weight<VEC>(p.w, i, p.dt_w, offset, w);
#pragma unroll
            for (int j = 0; j < VEC; ++j) a[k][j] *= rs * w[j] * (first ? 1.f : g[k][j]);
            store_vec<T, VEC>(y + i, a[k]);
        }
    }
}

template <typename T, typename TR, int VEC, int ITEMS>
__global__ void __launch_bounds__(kMaxThreads<VEC>) residual_norm_kernel(const ResidualNormParams p, int lanes) {
    __shared__ float red[2][32];
    const int per_cta = blockDim.x / lanes;
    const int64_t r = (int64_t)blockIdx.x * per_cta + threadIdx.x / lanes;
    const int t = threadIdx.x % lanes;
    const bool live = r < p.N;
    const int64_t n = live ? r : 0;
    const T *y = reinterpret_cast<const T *>(p.y) + n * p.ys;
    const T *z = reinterpret_cast<const T *>(p.z) + n * p.zs;
    const TR *x = reinterpret_cast<const TR *>(p.x) + n * p.D;
    const int act = p.flags & 0xF;
    const float offset = (p.flags & GDN_NORM_UNIT_OFFSET) ? 1.f : 0.f;
    float u[ITEMS][VEC], g[ITEMS][VEC], a[ITEMS][VEC];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = (k * lanes + t) * VEC;
        const bool in = live && i < p.D;
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[k][j] = 0.f, g[k][j] = 0.f, a[k][j] = 0.f;
        if (in) load_vec<T, VEC>(y + i, u[k]);
        if (in && act != GDN_GATE_NONE) load_vec<T, VEC>(z + i, g[k]);
        if (in && p.x != nullptr) load_vec<TR, VEC>(x + i, a[k]);
    }
    float rs = 1.f;
    if (p.w_post != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k)
#pragma unroll
            for (int j = 0; j < VEC; ++j) ss = fmaf(u[k][j], u[k][j], ss);
        rs = 1.f / sqrtf(row_sum(ss, lanes, red[0]) / (float)p.D + p.eps);
    }
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = (k * lanes + t) * VEC;
        if (live && i < p.D) {
            if (p.w_post != nullptr) {
                float w[VEC];
                load_weight<VEC>(p.w_post, i, p.dt_w, offset, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) u[k][j] *= rs * w[j];
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (act != GDN_GATE_NONE) u[k][j] *= activation<T>(g[k][j], act);
                a[k][j] = fmaf(p.scale, u[k][j], a[k][j]);
                ss = fmaf(a[k][j], a[k][j], ss);
            }
            if (p.x_out != nullptr) store_vec<TR, VEC>(reinterpret_cast<TR *>(p.x_out) + n * p.D + i, a[k]);
        }
    }
    if (p.out == nullptr) return;
    rs = 1.f / sqrtf(row_sum(ss, lanes, red[1]) / (float)p.D + p.eps);
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
    int items = 2;
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

template <typename T>
cudaError_t launch_gated_t(const GatedNormParams &p, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    // 16-byte vectors where every row of x, z and out starts on 16 bytes
    const bool vec = p.d % V == 0 && p.xs % V == 0 && p.os % V == 0 && (p.z == nullptr || p.zs % V == 0) &&
                     aligned16(p.x) && aligned16(p.z) && aligned16(p.out);
    const Spread s = spread(p.d, vec ? V : 1);
    const int64_t rows = p.N * p.H, per = s.threads / s.lanes;
    const unsigned grid = (unsigned)((rows + per - 1) / per);
    return with_items(s.items, [&](auto items) {
        constexpr int I = decltype(items)::value;
        if (vec) gated_norm_kernel<T, V, (I > 8 ? 8 : I)><<<grid, s.threads, 0, stream>>>(p, s.lanes);
        else gated_norm_kernel<T, 1, I><<<grid, s.threads, 0, stream>>>(p, s.lanes);
        return cudaGetLastError();
    });
}

template <typename T, typename TR>
cudaError_t launch_residual_t(const ResidualNormParams &p, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool vec = p.D % V == 0 && p.ys % V == 0 && (p.z == nullptr || p.zs % V == 0) && aligned16(p.y) &&
                     aligned16(p.z) && aligned16(p.x) && aligned16(p.x_out) && aligned16(p.out);
    const Spread s = spread(p.D, vec ? V : 1);
    const int64_t per = s.threads / s.lanes;
    const unsigned grid = (unsigned)((p.N + per - 1) / per);
    return with_items(s.items, [&](auto items) {
        constexpr int I = decltype(items)::value;
        if (vec) residual_norm_kernel<T, TR, V, (I > 8 ? 8 : I)><<<grid, s.threads, 0, stream>>>(p, s.lanes);
        else residual_norm_kernel<T, TR, 1, I><<<grid, s.threads, 0, stream>>>(p, s.lanes);
        return cudaGetLastError();
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
