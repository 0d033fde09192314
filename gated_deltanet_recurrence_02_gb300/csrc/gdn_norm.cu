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
// Both are bound by HBM where rows are vectors: every input element is read once, kept
// in registers in fp32 across the reductions, and every output element written once.  A
// row is spread over a group of threads (part of a warp, or a whole CTA), each holding
// ITEMS 16-byte vectors of it.  Sums of squares are fp32; h is formed from the unrounded
// x'; each output is rounded once.  What a single wave of CTAs over the rows leaves on
// the table is its start and end; 16-bit elements cost their conversions and the gate's
// exponential and reciprocal besides, so the gated norm's time follows its instructions.
// Measured:
//   gated, 4100 x 32 x 128 bf16   18.5 to 20.1 us (5.0 to 5.4 TB/s, 0.74 to 0.80 of the measured
//     copy bandwidth; 22.7 with a division a row and one element an instruction, 26.5
//     with the next row in registers instead of the ring below); fp32 35 us (5.8 TB/s)
//   residual, 4100 x 4096 bf16, fp32 residual, gate, both norms   45 us (5.2 TB/s, 0.77;
//     52 with the ring of per-thread copies that shorter rows use); 2050 x 8192: 53 us;
//     4100 x 2048: 21 us (5.6 TB/s); 10000 x 1024 bf16, bf16 residual: 22.5 us (4.5 TB/s)
// Rows that are not aligned to 16 bytes (odd widths, odd strides) are read and written an
// element a lane: 4100 x 2047 bf16, fp32 residual, gate
// 37 us (floor 17), 2000 x 32 x 129 23 us (7).
#include <atomic>

#include "gdn_internal.cuh"
#include "tc_ptx.cuh"

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

// Elementwise arithmetic on a vector, by fp32 pairs (one instruction for two elements:
// 16-bit norms are bound by their instructions before HBM).
__device__ __forceinline__ float2 pair(const float *x) { return make_float2(x[0], x[1]); }
__device__ __forceinline__ void put(float *x, float2 v) { x[0] = v.x, x[1] = v.y; }
template <int VEC>
__device__ __forceinline__ void mul(float (&a)[VEC], const float (&b)[VEC]) {
    if constexpr (VEC == 1) {
        a[0] *= b[0];
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) put(a + j, __fmul2_rn(pair(a + j), pair(b + j)));
    }
}
template <int VEC>
__device__ __forceinline__ void mul(float (&a)[VEC], float b) {
    if constexpr (VEC == 1) {
        a[0] *= b;
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) put(a + j, __fmul2_rn(pair(a + j), make_float2(b, b)));
    }
}
// a <- b c + a
template <int VEC>
__device__ __forceinline__ void add_mul(float (&a)[VEC], float b, const float (&c)[VEC]) {
    if constexpr (VEC == 1) {
        a[0] = fmaf(b, c[0], a[0]);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 2)
            put(a + j, __ffma2_rn(make_float2(b, b), pair(c + j), pair(a + j)));
    }
}
// The sum of squares, in two halves.
template <int VEC>
__device__ __forceinline__ void add_squares(float2 &ss, const float (&a)[VEC]) {
    if constexpr (VEC == 1) {
        ss.x = fmaf(a[0], a[0], ss.x);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) ss = __ffma2_rn(pair(a + j), pair(a + j), ss);
    }
}

// 1 / (1 + e^-z) by the base-2 exponential and the reciprocal of the PTX ISA
// (relative errors 2^-22 and 2^-23).  For 16-bit values the rounding of z log2 e is as
// far below their own as those; fp32 takes its rest along.  act(z), in place; the
// branches are the same for every thread.
template <typename T, int VEC>
__device__ __forceinline__ void activate(float (&z)[VEC], int act) {
    float s[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[j] = z[j];
    mul(s, -1.4426950408889634f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(s[j]));
        if constexpr (sizeof(T) == 4) {
            const float rest = fmaf(-1.4426950408889634f, z[j], -s[j]);
            const float more = e * (0.6931471805599453f * rest);
            e = fabsf(s[j]) < 126.f ? e + more : e;  // (no rest beside an infinite e or z)
        }
        s[j] = e;
    }
    // (a quarter of 1 + e^-z: its reciprocal is a normal number wherever e^-z is finite)
    if constexpr (VEC == 1) {
        s[0] = fmaf(s[0], 0.25f, 0.25f);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 2)
            put(s + j, __ffma2_rn(pair(s + j), make_float2(0.25f, 0.25f), make_float2(0.25f, 0.25f)));
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(s[j]));
    mul(s, 0.25f);
    if (act == GDN_GATE_SILU) {
        mul(z, s);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) z[j] = s[j];
    }
}

// Sum over the row's group of threads: `lanes` (a power of two) threads of a
// warp, or, with lanes > 32, all THREADS of the CTA.  red: a float for each warp,
// another buffer in every second call.  `any` (a whole CTA's rows only) becomes whether
// it was set in any thread.
template <int THREADS>
__device__ __forceinline__ float row_sum(float x, int lanes, float *red, bool *any = nullptr) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lanes <= 32) return x;
    constexpr int W = THREADS / 32;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    if (any != nullptr) *any = __syncthreads_or(*any) != 0;
    else __syncthreads();
    float s = red[threadIdx.x & (W - 1)];
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// Rows on their way.  With vectors, each thread copies its own 16-byte pieces of
// its next rows to shared memory, DEPTH rows deep (cp.async: no other thread
// reads them, so no barrier stands between copy and use); without, the next row
// waits in registers.  NP: pieces of a row a thread.
template <int NP, int THREADS>
struct Ring {
    static constexpr int kRow = NP * THREADS * 16;
    // (most of a CTA's ring: two CTAs an SM)
    static constexpr int DEPTH = 98304 / kRow > 4 ? 4 : 98304 / kRow < 1 ? 1 : 98304 / kRow;
    static constexpr int kBytes = DEPTH * kRow;
    uint32_t mine;
    __device__ __forceinline__ Ring(const uint4 *base)
        : mine(static_cast<uint32_t>(__cvta_generic_to_shared(base + threadIdx.x))) {}
    __device__ __forceinline__ void copy(int slot, int piece, const void *src) const {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine + slot * kRow + piece * THREADS * 16), "l"(src)
                     : "memory");
    }
    __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // all but the last DEPTH - 1 rows copied
    __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory"); }
    template <typename R>
    __device__ __forceinline__ void get(int slot, int piece, R &raw) const {
#pragma unroll
        for (int k = 0; k < R::kPacks; ++k) {
            uint4 &u = *reinterpret_cast<uint4 *>(&raw.v[k]);
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                         : "r"(mine + slot * kRow + (piece + k) * THREADS * 16)
                         : "memory");
        }
    }
    __device__ __forceinline__ static int next(int slot) { return slot + 1 == DEPTH ? 0 : slot + 1; }
};

// CTAs an SM at least, which is a limit of registers: 64 a thread, 80 or 128 where a row
// has more elements a thread (4100 x 4095 bf16, eight of them: 90 us with 64 and spills,
// 71).  The widest rows still spill: the gated norm's of more than 16 elements a thread
// some 340 (16-bit) and 1060 bytes (fp32) a thread, and unaligned rows of more than 8192
// elements, where 1024 threads leave 64 registers each, 780 to 1090.
constexpr int ctas_of(int vec, int items, int threads) {
    return vec * items > 8 ? 1 : (vec == 1 && items > 5 ? 768 : 1024) / threads;
}

template <typename T, int VEC, int ITEMS, int THREADS>
__global__ void __launch_bounds__(THREADS, ctas_of(VEC, ITEMS, THREADS)) gated_norm_kernel(const GatedNormParams p, int lanes) {
    __shared__ float red[2][32];
    extern __shared__ uint4 ring_smem[];
    using R = Ring<2 * ITEMS, THREADS>;
    const R ring(ring_smem);
    const int per_cta = THREADS / lanes;
    const unsigned rows = (unsigned)(p.N * p.H), H = (unsigned)p.H;
    const int t = threadIdx.x % lanes;
    const int act = p.gate & 0xF;
    const bool first = (p.gate & GDN_GATE_FIRST) != 0;
    const float offset = (p.gate & GDN_NORM_UNIT_OFFSET) ? 1.f : 0.f;
    const float inv_d = 1.f / (float)p.d;
    // the thread's columns, and so its weights, are the same in every row
    float w[ITEMS][VEC];
    Raw<T, VEC> nx[ITEMS], nz[ITEMS];
    bool in[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = (k * lanes + t) * VEC;
        in[k] = i < p.d;
        nx[k].clear();
        nz[k].clear();
        if (in[k]) load_weight<VEC>(p.w, i, p.dt_w, offset, w[k]);
    }
    // (every thread of a CTA takes as many turns: the sums are taken together)
    const unsigned step = gridDim.x * per_cta;
    unsigned base = blockIdx.x * per_cta;
    const unsigned step_n = step / H, step_h = step - step_n * H;
    struct Row {  // head h of token n (h d may pass 32 bits)
        unsigned r, n, h;
    };
    auto advance = [&](Row &x) {
        x.r += step;
        x.n += step_n;
        x.h += step_h;
        if (x.h >= H) x.h -= H, ++x.n;
    };
    Row out;  // the next one to finish, and to fetch
    out.r = base + threadIdx.x / lanes;
    out.n = out.r / H;
    out.h = out.r - out.n * H;
    Row in_row = out;
    auto fetch = [&](int slot) {  // unless it is past the last
        if (in_row.r >= rows) return;
        const T *x = reinterpret_cast<const T *>(p.x) + (int64_t)in_row.n * p.xs + (uint64_t)in_row.h * (unsigned)p.d + t * VEC;
        const T *z = reinterpret_cast<const T *>(p.z) + (int64_t)in_row.n * p.zs + (uint64_t)in_row.h * (unsigned)p.d + t * VEC;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            if (in[k]) {
                if constexpr (VEC > 1) {
                    ring.copy(slot, 2 * k, x + k * lanes * VEC);
                    if (act != GDN_GATE_NONE) ring.copy(slot, 2 * k + 1, z + k * lanes * VEC);
                } else {
                    nx[k].load(x + k * lanes);
                    if (act != GDN_GATE_NONE) nz[k].load(z + k * lanes);
                }
            }
        }
    };
    int parity = 0, slot = 0;
    for (int k = 0; k < (VEC > 1 ? R::DEPTH - 1 : 1); ++k) {
        fetch(k);
        advance(in_row);
        if constexpr (VEC > 1) ring.commit();
    }
    for (; base < rows; base += step, parity ^= 1, advance(out)) {
        if constexpr (VEC > 1) {
            fetch(slot == 0 ? R::DEPTH - 1 : slot - 1);
            advance(in_row);
            ring.commit();
            ring.wait();
#pragma unroll
            for (int k = 0; k < ITEMS; ++k)
                if (in[k]) {
                    ring.get(slot, 2 * k, nx[k]);
                    if (act != GDN_GATE_NONE) ring.get(slot, 2 * k + 1, nz[k]);
                }
            slot = R::next(slot);
        }
        float a[ITEMS][VEC], g[ITEMS][VEC];
        float2 ss2 = make_float2(0.f, 0.f);
        // (columns past the row are zeros; rows past the last are not stored)
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            nx[k].get(a[k]);
            if (act != GDN_GATE_NONE) {
                nz[k].get(g[k]);
                activate<T, VEC>(g[k], act);
                if (first) mul(a[k], g[k]);
            }
            add_squares(ss2, a[k]);
        }
        if constexpr (VEC == 1) {
            fetch(0);
            advance(in_row);
        }
        const float ss = row_sum<THREADS>(ss2.x + ss2.y, lanes, red[parity]);
        const float rs = rsqrtf(fmaf(ss, inv_d, p.eps));
        if (out.r < rows) {
            T *y = reinterpret_cast<T *>(p.out) + (int64_t)out.n * p.os + (uint64_t)out.h * (unsigned)p.d + t * VEC;
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                if (in[k]) {
                    mul(a[k], rs);
                    mul(a[k], w[k]);
                    if (act != GDN_GATE_NONE && !first) mul(a[k], g[k]);
                    store_vec<T, VEC>(y + k * lanes * VEC, a[k]);
                }
            }
        }
    }
}

// A weight's vector for the thread's columns: kept in registers where they are few
// enough, else read again for every row: from shared memory, in fp32, where the CTA's
// rows are short (`share`; 10000 x 1024 bf16: 22.5 us, 26.6 with loads and conversions
// from L1), else from L1.
template <int VEC, int ITEMS>
struct Weights {
    static constexpr bool kKept = VEC * ITEMS <= 8;
    float w[kKept ? ITEMS : 1][VEC];
    __device__ __forceinline__ void keep(const void *p, int i, int dt, float offset, int k) {
        if constexpr (kKept) load_weight<VEC>(p, i, dt, offset, w[k]);
    }
    __device__ __forceinline__ const float (&at(const void *p, int i, int dt, float offset, int k))[VEC] {
        if constexpr (kKept) return w[k];
        load_weight<VEC>(p, i, dt, offset, w[0]);
        return w[0];
    }
    // All D weights by the whole CTA, element 4 e of vector v at [128 e + v].
    template <int THREADS>
    __device__ __forceinline__ static void share(float4 *s, const void *p, int D, int dt, float offset) {
        for (int i = threadIdx.x; i < D / 4; i += THREADS) {
            float x[4];
            load_weight<4>(p, 4 * i, dt, offset, x);
            s[i % (VEC / 4) * 128 + i / (VEC / 4)] = make_float4(x[0], x[1], x[2], x[3]);
        }
    }
    __device__ __forceinline__ const float (&at(const float4 *s, int v))[VEC] {
#pragma unroll
        for (int e = 0; e < VEC / 4; ++e) {
            const float4 f = s[128 * e + v];
            w[0][4 * e] = f.x, w[0][4 * e + 1] = f.y, w[0][4 * e + 2] = f.z, w[0][4 * e + 3] = f.w;
        }
        return w[0];
    }
};

template <typename T, typename TR, int VEC, int ITEMS, int THREADS>
__global__ void __launch_bounds__(THREADS, ctas_of(VEC, ITEMS, THREADS)) residual_norm_kernel(const ResidualNormParams p, int lanes) {
    __shared__ float red[2][32];
    extern __shared__ uint4 ring_smem[];
    constexpr int XP = Raw<TR, VEC>::kPacks, NP = 2 + XP;
    using R = Ring<NP * ITEMS, THREADS>;
    const R ring(ring_smem);
    const int per_cta = THREADS / lanes, t = threadIdx.x % lanes;
    const int act = p.flags & 0xF;
    const float offset = (p.flags & GDN_NORM_UNIT_OFFSET) ? 1.f : 0.f;
    const float inv_d = 1.f / (float)p.D;
    const bool post = p.w_post != nullptr;
    Raw<T, VEC> ny[ITEMS], nz[ITEMS];
    Raw<TR, VEC> nx[ITEMS];
    using W = Weights<VEC, ITEMS>;
    W w_post, w_pre;
    constexpr bool kShared = VEC > 1 && !W::kKept;
    __shared__ float4 shared_w[kShared ? 2 : 1][kShared ? 256 : 1];
    if constexpr (kShared) {
        if (post) W::template share<THREADS>(shared_w[0], p.w_post, p.D, p.dt_w, offset);
        W::template share<THREADS>(shared_w[1], p.w_pre, p.D, p.dt_w, offset);
        __syncthreads();
    }
    bool in[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = (k * lanes + t) * VEC;
        in[k] = i < p.D;
        ny[k].clear();
        nz[k].clear();
        nx[k].clear();
        if (in[k]) {
            if (post) w_post.keep(p.w_post, i, p.dt_w, offset, k);
            w_pre.keep(p.w_pre, i, p.dt_w, offset, k);
        }
    }
    auto fetch = [&](int64_t n, int slot) {
        const T *y = reinterpret_cast<const T *>(p.y) + n * p.ys + t * VEC;
        const T *z = reinterpret_cast<const T *>(p.z) + n * p.zs + t * VEC;
        const TR *x = reinterpret_cast<const TR *>(p.x) + n * p.D + t * VEC;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            if (in[k]) {
                const int i = k * lanes * VEC;
                if constexpr (VEC > 1) {
                    ring.copy(slot, NP * k, y + i);
                    if (act != GDN_GATE_NONE) ring.copy(slot, NP * k + 1, z + i);
                    if (p.x != nullptr)
#pragma unroll
                        for (int e = 0; e < XP; ++e) ring.copy(slot, NP * k + 2 + e, x + i + e * (VEC / XP));
                } else {
                    ny[k].load(y + i);
                    if (act != GDN_GATE_NONE) nz[k].load(z + i);
                    if (p.x != nullptr) nx[k].load(x + i);
                }
            }
        }
    };
    // (every thread of a CTA takes as many turns: the sums are taken together)
    const int64_t step = (int64_t)gridDim.x * per_cta;
    int64_t n = (int64_t)blockIdx.x * per_cta + threadIdx.x / lanes, base = (int64_t)blockIdx.x * per_cta;
    int slot = 0;
    if constexpr (VEC > 1) {
        for (int k = 0; k < R::DEPTH - 1; ++k) {
            if (n + k * step < p.N) fetch(n + k * step, k);
            ring.commit();
        }
    } else if (n < p.N) {
        fetch(n, 0);
    }
    for (; base < p.N; base += step, n += step) {
        if constexpr (VEC > 1) {
            const int64_t ahead = n + (R::DEPTH - 1) * step;
            if (ahead < p.N) fetch(ahead, slot == 0 ? R::DEPTH - 1 : slot - 1);
            ring.commit();
            ring.wait();
#pragma unroll
            for (int k = 0; k < ITEMS; ++k)
                if (in[k]) {
                    ring.get(slot, NP * k, ny[k]);
                    if (act != GDN_GATE_NONE) ring.get(slot, NP * k + 1, nz[k]);
                    if (p.x != nullptr) ring.get(slot, NP * k + 2, nx[k]);
                }
            slot = R::next(slot);
        }
        float u[ITEMS][VEC], a[ITEMS][VEC];
        float2 ss = make_float2(0.f, 0.f);
        // (columns past the row are zeros; rows past the last are not stored)
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            ny[k].get(u[k]);
            nx[k].get(a[k]);
            if (post) add_squares(ss, u[k]);
            if (act != GDN_GATE_NONE) {
                float g[VEC];
                nz[k].get(g);
                activate<T, VEC>(g, act);
                mul(u[k], g);
            }
        }
        if constexpr (VEC == 1)
            if (n + step < p.N) fetch(n + step, 0);
        float rs = p.scale;
        if (post) rs *= rsqrtf(fmaf(row_sum<THREADS>(ss.x + ss.y, lanes, red[0]), inv_d, p.eps));
        ss = make_float2(0.f, 0.f);
        const bool live = n < p.N;
        TR *x_out = reinterpret_cast<TR *>(p.x_out) + n * p.D + t * VEC;
        T *out = reinterpret_cast<T *>(p.out) + n * p.D + t * VEC;
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = k * lanes * VEC;
            if (live && in[k]) {
                if (post) {
                    const float(&w)[VEC] = kShared ? w_post.at(shared_w[0], k * lanes + t)
                                                   : w_post.at(p.w_post, i + t * VEC, p.dt_w, offset, k);
                    mul(u[k], w);
                }
                add_mul(a[k], rs, u[k]);
                add_squares(ss, a[k]);
                if (p.x_out != nullptr) store_vec<TR, VEC>(x_out + i, a[k]);
            }
        }
        if (p.out != nullptr) {
            rs = rsqrtf(fmaf(row_sum<THREADS>(ss.x + ss.y, lanes, red[1]), inv_d, p.eps));
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int i = k * lanes * VEC;
                if (live && in[k]) {
                    const float(&w)[VEC] = kShared ? w_pre.at(shared_w[1], k * lanes + t)
                                                   : w_pre.at(p.w_pre, i + t * VEC, p.dt_w, offset, k);
                    mul(a[k], rs);
                    mul(a[k], w);
                    store_vec<T, VEC>(out + i, a[k]);
                }
            }
        }
        // with only one of the two sums no barrier stands between this one and the
        // next turn's
        if (lanes > 32 && (!post || p.out == nullptr)) __syncthreads();
    }
}

// residual_norm of rows longer than a warp's 128 vectors: a CTA a row, its next rows
// on their way to shared memory by bulk copies, `stages` deep.  A bulk copy costs
// one thread a few instructions a row, where per-thread copies cost every thread
// more than the norm's own arithmetic.  Rows are multiples of 16 bytes.
template <typename T, typename TR, int ITEMS, int THREADS>
__global__ void __launch_bounds__(THREADS, ITEMS == 1 ? 1024 / THREADS : 1)
residual_row_kernel(const ResidualNormParams p, int stages) {
    constexpr int VEC = 16 / (int)sizeof(T);
    __shared__ float red[2][32];
    __shared__ uint64_t full[4];
    extern __shared__ uint4 ring_smem[];
    uint8_t *sm = reinterpret_cast<uint8_t *>(ring_smem);
    const int t = threadIdx.x, D = p.D;
    const int act = p.flags & 0xF;
    const float offset = (p.flags & GDN_NORM_UNIT_OFFSET) ? 1.f : 0.f;
    const float inv_d = 1.f / (float)D;
    const bool post = p.w_post != nullptr;
    const bool wide = (reinterpret_cast<uintptr_t>(p.x_out) & 31) == 0;
    // a stage: y, then the gate and the residual where there are any
    const uint32_t yb = (uint32_t)D * sizeof(T), zb = act != GDN_GATE_NONE ? yb : 0u;
    const uint32_t xb = p.x != nullptr ? (uint32_t)D * sizeof(TR) : 0u, bytes = yb + zb + xb;
    if (t == 0) {
        for (int s = 0; s < stages; ++s) tc::mbar_init(&full[s], 1);
        tc::fence_mbar_init();
    }
    Weights<VEC, ITEMS> w_post, w_pre;
    bool in[ITEMS];
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
        const int i = (k * THREADS + t) * VEC;
        in[k] = i < D;
        if (in[k]) {
            if (post) w_post.keep(p.w_post, i, p.dt_w, offset, k);
            w_pre.keep(p.w_pre, i, p.dt_w, offset, k);
        }
    }
    __syncthreads();
    auto issue = [&](int64_t n, int s) {  // one thread
        uint8_t *st = sm + s * bytes;
        tc::mbar_arrive_expect_tx(&full[s], bytes);
        tc::bulk_load(st, reinterpret_cast<const T *>(p.y) + n * p.ys, yb, &full[s]);
        if (zb) tc::bulk_load(st + yb, reinterpret_cast<const T *>(p.z) + n * p.zs, zb, &full[s]);
        if (xb) tc::bulk_load(st + yb + zb, reinterpret_cast<const TR *>(p.x) + n * D, xb, &full[s]);
    };
    const int64_t step = gridDim.x;
    int64_t n = blockIdx.x;
    if (t == 0)
        for (int s = 0; s < stages; ++s)
            if (n + s * step < p.N) issue(n + s * step, s);
    int s = 0, phase = 0;
    bool late = false;  // a copy did not come in time, as any thread saw it
    for (; n < p.N; n += step) {
        late = !tc::mbar_wait(&full[s], phase, p.wait_ns);
        const uint8_t *st = sm + s * bytes;
        float u[ITEMS][VEC], a[ITEMS][VEC];
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = (k * THREADS + t) * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[k][j] = 0.f, a[k][j] = 0.f;
            if (!in[k]) continue;
            load_vec<T, VEC>(reinterpret_cast<const T *>(st) + i, u[k]);
            if (xb) load_vec<TR, VEC>(reinterpret_cast<const TR *>(st + yb + zb) + i, a[k]);
            if (post) add_squares(ss, u[k]);
            if (zb) {
                float g[VEC];
                load_vec<T, VEC>(reinterpret_cast<const T *>(st + yb) + i, g);
                activate<T, VEC>(g, act);
                mul(u[k], g);
            }
        }
        float rs = p.scale;
        if (post) rs *= rsqrtf(fmaf(row_sum<THREADS>(ss.x + ss.y, THREADS, red[0], &late), inv_d, p.eps));
        else late = __syncthreads_or(late) != 0;
        if (late) break;  // the whole CTA, before any of the row is written
        // every thread has read the stage
        if (t == 0 && n + stages * step < p.N) issue(n + stages * step, s);
        ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < ITEMS; ++k) {
            const int i = (k * THREADS + t) * VEC;
            if (!in[k]) continue;
            if (post) {
                const float(&w)[VEC] = w_post.at(p.w_post, i, p.dt_w, offset, k);
                mul(u[k], w);
            }
            add_mul(a[k], rs, u[k]);
            add_squares(ss, a[k]);
            if (p.x_out != nullptr) {
                TR *dst = reinterpret_cast<TR *>(p.x_out) + n * D + i;
                if constexpr (sizeof(TR) * VEC == 32) {
                    if (wide)
                        st8_wide(dst, make_float2(a[k][0], a[k][1]), make_float2(a[k][2], a[k][3]),
                                 make_float2(a[k][4], a[k][5]), make_float2(a[k][6], a[k][7]));
                    else
                        store_vec<TR, VEC>(dst, a[k]);
                } else {
                    store_vec<TR, VEC>(dst, a[k]);
                }
            }
        }
        if (p.out != nullptr) {
            rs = rsqrtf(fmaf(row_sum<THREADS>(ss.x + ss.y, THREADS, red[1]), inv_d, p.eps));
#pragma unroll
            for (int k = 0; k < ITEMS; ++k) {
                const int i = (k * THREADS + t) * VEC;
                if (!in[k]) continue;
                const float(&w)[VEC] = w_pre.at(p.w_pre, i, p.dt_w, offset, k);
                mul(a[k], rs);
                mul(a[k], w);
                store_vec<T, VEC>(reinterpret_cast<T *>(p.out) + n * D + i, a[k]);
            }
        } else if (post) {
            __syncthreads();  // red[0] is written again in the next turn
        }
        if (++s == stages) s = 0, phase ^= 1;
    }
    if (late && t == 0) {
        atomicOr(p.err, (uint32_t)GDN_DEVERR_TIMEOUT);
        // the copies in flight, of this row and of those after it, must land before the CTA ends
        for (int k = 0; k < stages && n < p.N; ++k, n += step) {
            tc::mbar_wait(&full[s], phase, kDefaultWaitNs / 8);
            if (++s == stages) s = 0, phase ^= 1;
        }
    }
}

// How a row of `width` elements is spread over threads of ITEMS vectors each.
// Rows of up to 32 vectors take the smallest power of two of lanes of one vector
// each, so several rows share a warp; up to 128 (single elements: 512, where a CTA's
// two barriers a row made 4100 x 4 rows of 257 take 43 us, now 23) a warp; longer
// ones a whole CTA.
struct Spread {
    int lanes, threads, items;
};
Spread spread(int width, int vec) {
    const int nv = (width + vec - 1) / vec;
    if (nv <= (vec > 1 ? 128 : 512)) {
        int lanes = 1;
        while (lanes < 32 && lanes < nv) lanes *= 2;
        return {lanes, 256, (nv + lanes - 1) / lanes};
    }
    if (vec > 1 && nv <= 256) return {256, 256, 1};
    const int threads = nv > 16 * 512 ? 1024 : 512;
    return {threads, threads, (nv + threads - 1) / threads};
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// CTAs that run at once, asked once a device; 0 if the question failed.
template <auto Kern>
unsigned resident(int threads, int bytes) {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int c = cache[dev].load(std::memory_order_relaxed);
    if (c == 0) {
        if (bytes > 0 && set_smem_once<Kern>(bytes) != cudaSuccess) return 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&c, Kern, threads, bytes) != cudaSuccess || c < 1) return 0;
        c *= sm_count_of_current_device();
        cache[dev].store(c, std::memory_order_relaxed);
    }
    return (unsigned)c;
}
template <auto Kern, int BYTES, typename P>
cudaError_t launch_rows(const P &p, const Spread &s, int64_t rows, cudaStream_t stream) {
    const int64_t per = s.threads / s.lanes, ctas = (rows + per - 1) / per;
    const unsigned most = resident<Kern>(s.threads, BYTES);
    if (most == 0) return cudaErrorInvalidConfiguration;
    Kern<<<ctas < most ? (unsigned)ctas : most, s.threads, BYTES, stream>>>(p, s.lanes);
    return cudaGetLastError();
}

constexpr int kRowSmem = 204800;  // a multiprocessor's shared memory for rows
constexpr int kSmSmem = 228 * 1024;  // all of it (a CTA takes 1 KB and its barriers besides its rows)

template <int I, int TH>
struct Shape {
    static constexpr int items = I, threads = TH;
};
// Calls f with the spread's threads and the least items of those built that hold its
// row as constants.  A row of vectors has at most 32 elements a thread, so never more
// than MOST vectors, in powers of two; single elements come in finer steps, as their
// loads and stores are what such rows cost (2000 x 32 x 129 bf16: 23 us as five a lane,
// 35 as eight).
template <int MOST, int THREADS, int I, typename F>
cudaError_t with_items(int items, F f) {
    constexpr int next = MOST > 8 && (I == 2 || I == 4) ? I + 1 : I == 3 ? 4 : I == 5 ? 6 : I == 6 ? 8 : MOST > 8 && I == 8 ? 12 : I == 12 ? 16 : 2 * I;
    if constexpr (next <= MOST && (THREADS == 512 || MOST > 8 || next <= 4)) {
        if (items > I) return with_items<MOST, THREADS, next>(items, f);
    }
    return f(Shape<I, THREADS>{});
}
template <int MOST, typename F>
cudaError_t with_shape(const Spread &s, F f) {
    if (s.threads == 256) return with_items<MOST, 256, 1>(s.items, f);
    if constexpr (MOST > 8)
        if (s.threads == 1024) return f(Shape<16, 1024>{});
    return with_items<MOST, 512, 1>(s.items, f);
}

template <typename T>
cudaError_t launch_gated_t(const GatedNormParams &p, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    // 16-byte vectors where every row of x, z and out starts on 16 bytes
    const bool vec = p.d % V == 0 && p.xs % V == 0 && p.os % V == 0 && (p.z == nullptr || p.zs % V == 0) &&
                     aligned16(p.x) && aligned16(p.z) && aligned16(p.out) && aligned16(p.w);
    const Spread s = spread(p.d, vec ? V : 1);
    if (vec)
        return with_shape<32 / V>(s, [&](auto shape) {
            using S = decltype(shape);
            return launch_rows<gated_norm_kernel<T, V, S::items, S::threads>, Ring<2 * S::items, S::threads>::kBytes>(
                p, s, p.N * p.H, stream);
        });
    return with_shape<16>(s, [&](auto shape) {
        using S = decltype(shape);
        return launch_rows<gated_norm_kernel<T, 1, S::items, S::threads>, 0>(p, s, p.N * p.H, stream);
    });
}

template <typename T, typename TR>
cudaError_t launch_residual_t(const ResidualNormParams &p, cudaStream_t stream) {
    constexpr int V = 16 / (int)sizeof(T);
    const bool vec = p.D % V == 0 && p.ys % V == 0 && (p.z == nullptr || p.zs % V == 0) && aligned16(p.y) &&
                     aligned16(p.z) && aligned16(p.x) && aligned16(p.x_out) && aligned16(p.out) &&
                     aligned16(p.w_post) && aligned16(p.w_pre);
    const Spread s = spread(p.D, vec ? V : 1);
    if (vec && s.lanes > 32)
        return with_shape<32 / V>(s, [&](auto shape) {
            using S = decltype(shape);
            constexpr auto kern = residual_row_kernel<T, TR, S::items, S::threads>;
            // as many CTAs an SM as make 1024 threads, where two rows fit each of two; as
            // many stages, up to four, as fit each of them, so that all run at once (4100 x
            // 2048 bf16 with a gate and an fp32 residual: 20.8 us with three stages, 26.7 with
            // four, where a quarter of the CTAs are a second wave)
            const int row = p.D * (int)(sizeof(T) * (p.z != nullptr ? 2 : 1) + (p.x != nullptr ? sizeof(TR) : 0));
            const int per_sm = row <= kRowSmem / 4 ? 1024 / S::threads : 1;
            const int most = per_sm > 2 ? kSmSmem / per_sm - 2048 : kRowSmem / per_sm;
            const int stages = most / row > 4 ? 4 : most / row < 1 ? 1 : most / row;
            const cudaError_t e = set_smem_once<kern>(kRowSmem);
            if (e != cudaSuccess) return e;
            const int64_t ctas = (int64_t)sm_count_of_current_device() * per_sm;
            kern<<<(unsigned)(p.N < ctas ? p.N : ctas), S::threads, stages * row, stream>>>(p, stages);
            return cudaGetLastError();
        });
    if (vec)
        return with_shape<32 / V>(s, [&](auto shape) {
            using S = decltype(shape);
            if constexpr (S::threads > 256) {
                return cudaErrorInvalidConfiguration;  // (a CTA's row: above)
            } else {
                constexpr int NP = (2 + (sizeof(TR) > sizeof(T) ? 2 : 1)) * S::items;
                return launch_rows<residual_norm_kernel<T, TR, V, S::items, S::threads>, Ring<NP, S::threads>::kBytes>(
                    p, s, p.N, stream);
            }
        });
    return with_shape<16>(s, [&](auto shape) {
        using S = decltype(shape);
        return launch_rows<residual_norm_kernel<T, TR, 1, S::items, S::threads>, 0>(p, s, p.N, stream);
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
