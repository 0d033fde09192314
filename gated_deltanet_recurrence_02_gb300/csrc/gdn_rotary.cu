// gdn_rotary.cu -- rotary positions, alone and on the way into a paged cache.
//
// Pair i < R / 2 of a head, (x1, x2) = elements (i, i + R / 2), or (2 i, 2 i + 1) with
// GDN_ROTARY_PAIRS, of a token at position p on the pair's axis:
//     phi = p f_i,   y1 = x1 cos phi - x2 sin phi,   y2 = x2 cos phi + x1 sin phi
// The turn back (GDN_ROTARY_INVERSE) takes -phi.  Elements from R on are copied.
//
// Angles.  p f_i in fp32 is off by 2^-24 of itself, 0.06 rad at a position of a million.
// Here f_i / 2 pi is held as a 64-bit fraction of a turn, formed in double once per CTA
// and frequency; p times it, modulo 2^64, is the angle modulo a turn, exact but for the
// 2^-52 of the fraction's own rounding.  Of its upper 32 bits the distance from the nearest
// quarter of a turn goes to sincospi, as half turns.
//
// One pass: every element is read and written once, and bound by HBM.  A CTA takes a few
// tokens at a time: it starts to load their vectors (V elements, 16 bytes where alignment and
// widths allow, of both halves of V pairs), forms the cosines and sines of their angles in
// shared memory, once for all heads, while those are on their way, then turns and stores.
// On the device: 4100 tokens x 32 heads x 128, three axes, bf16, 13.1 us, 5.1 TB/s; 16
// packed prompts of 100 to 600 tokens, 32 and 8 heads, appended, 26.7 us, 5.1 TB/s; seven
// tokens 2.6 us, a launch.  Vectors as wide as alignment allows:
// with 8, 4, 2, 1 elements the prompts take 26, 34, 50, 82 us.
#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kCtas = 5;          // that an SM holds at once
constexpr int kInFlight = 2;      // vectors a thread
constexpr int kMaxTokens = 128;   // a CTA at a time
constexpr int kMaxAngles = 2048;  // of them together (but those of one token)

struct RotaryShape {
    int tokens;        // a CTA at a time
    int turned;        // vectors of a head that turn (with their second halves)
    Divisor per_token, per_head, per_half;
};

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T v[V];
};

template <typename T>
__device__ __forceinline__ T rounded(float x) {
    T y;
    st_out(&y, x);
    return y;
}

// Elements 2 q and 2 q + 1 of a vector in fp32, and back.
template <typename T, int V>
__device__ __forceinline__ float2 get2(const Vec<T, V> &x, int q) {
    return make_float2(ld_f(&x.v[2 * q]), ld_f(&x.v[2 * q + 1]));
}
template <int V>
__device__ __forceinline__ float2 get2(const Vec<__half, V> &x, int q) {
    return __half22float2(reinterpret_cast<const __half2 *>(x.v)[q]);
}
template <typename T, int V>
__device__ __forceinline__ void put2(Vec<T, V> &x, int q, float2 y) {
    st_out(&x.v[2 * q], y.x);
    st_out(&x.v[2 * q + 1], y.y);
}
template <int V>
__device__ __forceinline__ void put2(Vec<__half, V> &x, int q, float2 y) {
    reinterpret_cast<__half2 *>(x.v)[q] = __float22half2_rn(y);
}
template <int V>
__device__ __forceinline__ void put2(Vec<__nv_bfloat16, V> &x, int q, float2 y) {
    reinterpret_cast<__nv_bfloat162 *>(x.v)[q] = __float22bfloat162_rn(y);
}

// Where a token's keys and values go, and the position that turns them where none is given.
struct Place {
    int64_t at;  // elements into the pages, or -1: nowhere
    int pos;     // in the cache
    int row;     // its row, or -1: none
};

// By a whole warp: for packed rows a search with 32 probes a round (a binary search's loads
// wait for one another log2 B times).
__device__ Place place_of(const RotaryParams &p, int64_t n) {
    const int lane = threadIdx.x % 32;
    Place x{-1, 0, -1};
    int b, t, len;
    if (p.cu_seqlens == nullptr) {
        b = (int)((uint32_t)n / (uint32_t)p.T);
        t = (int)(n - (int64_t)b * p.T);
        len = p.T;
    } else {
        b = 0;
        int rows = p.B;  // the last row that starts at or before n is one of these, from b on
        while (rows > 1) {
            const int step = (rows + 31) / 32, probe = lane * step;
            const unsigned in = __ballot_sync(0xffffffffu, probe < rows && p.cu_seqlens[b + probe] <= n);
            const int last = in != 0 ? 31 - __clz(in) : 0;
            b += last * step;
            rows = min(step, rows - last * step);
        }
        long tok0;
        row_range(p.cu_seqlens, b, (int)p.N, tok0, len);
        if (n < tok0 || n >= tok0 + len) return x;
        t = (int)(n - tok0);
    }
    x.row = b;
    const int64_t pos = (int64_t)max(p.kv_lens[b], 0) - len + t;
    x.pos = (int)pos;
    if (pos < 0) return x;  // before the cache's first position: kept nowhere
    const uint32_t page = (uint32_t)pos / (uint32_t)p.page_size;
    int id = -1;
    if (page < (uint32_t)p.max_pages) id = p.page_table[(int64_t)b * p.max_pages + page];
    if (id < 0 || id >= p.num_pages) {
        atomicOr(p.err, (uint32_t)GDN_DEVERR_BAD_INDEX);
        return x;
    }
    x.at = id * p.page_stride + (pos - (int64_t)page * p.page_size) * p.slot_stride;
    return x;
}

// A thread's vector of the CTA's tokens: both halves of V pairs, or one that is copied.
template <typename T, int V>
struct Item {
    Vec<T, V> a, b;
    int t, h, w;  // token, head, vector of the head; t < 0: nothing
};

template <typename T, int V, bool PAIRS, bool APPEND>
__global__ void __launch_bounds__(kThreads, kCtas) rotary_kernel(const RotaryParams p, const RotaryShape s) {
    // Cosines and sines of a token's angles.  Two neighbouring pairs' together (c c s s), the
    // vectors of a head next to each other, so that lanes read them without bank conflicts.
    extern __shared__ float4 angle4[];  // [tokens][V / 2][turned]; V = 1: float2 [tokens][turned]
    float2 *angle2 = reinterpret_cast<float2 *>(angle4);
    __shared__ uint64_t turns[kRotaryMaxWidth / 2];
    __shared__ int axis[kRotaryMaxWidth / 2];
    __shared__ Place place[APPEND ? kMaxTokens : 1];
    const int half = p.R / 2;
    const int second = PAIRS ? V : half;  // from a vector's first half to its second
    for (int i = threadIdx.x; i < half; i += kThreads) {
        const double f = (double)p.inv_freq[i] * 0.15915494309189533577;  // 1 / 2 pi
        // (2^63 of a turn's fraction in [-1/2, 1/2], twice)
        turns[i] = (uint64_t)__double2ll_rn((f - rint(f)) * 9223372036854775808.0) << 1;
        int a = p.axes != nullptr ? p.axes[i] : 0;
        if (a < 0 || a >= p.A) {  // (an axis that is not there turns nothing)
            atomicOr(p.err, (uint32_t)GDN_DEVERR_BAD_INDEX);
            turns[i] = 0;
            a = 0;
        }
        axis[i] = a;
    }
    const int64_t step = (int64_t)gridDim.x * s.tokens;
    for (int64_t n0 = (int64_t)blockIdx.x * s.tokens; n0 < p.N; n0 += step) {
        const int tokens = (int)(p.N - n0 < s.tokens ? p.N - n0 : s.tokens);
        const uint32_t items = (uint32_t)tokens * s.per_token.d;
        // offset in its head of vector w
        auto offset = [&](int w) { return w < s.turned ? (PAIRS ? 2 * V * w : V * w) : p.R + V * (w - s.turned); };
        auto load = [&](uint32_t e, Item<T, V> &x) {
            x.t = -1;
            if (e >= items) return;
            x.t = (int)s.per_token.div(e);
            const uint32_t r = e - x.t * s.per_token.d;
            x.h = (int)s.per_head.div(r);
            x.w = (int)(r - x.h * s.per_head.d);
            const int64_t n = n0 + x.t;
            const T *src;
            if (!APPEND || x.h < p.Hq) src = reinterpret_cast<const T *>(p.q) + n * p.qs + x.h * p.d;
            else if (x.h < p.Hq + p.Hk) src = reinterpret_cast<const T *>(p.k) + n * p.ks + (x.h - p.Hq) * p.d;
            else src = reinterpret_cast<const T *>(p.v) + n * p.vs + (x.h - p.Hq - p.Hk) * p.d;
            src += offset(x.w);
            x.a = *reinterpret_cast<const Vec<T, V> *>(src);
            if (x.w < s.turned) x.b = *reinterpret_cast<const Vec<T, V> *>(src + second);
        };
        auto finish = [&](Item<T, V> &x) {
            if (x.t < 0) return;
            T *dst;
            if (!APPEND || x.h < p.Hq) {
                if (APPEND && place[x.t].row < 0) return;
                dst = reinterpret_cast<T *>(p.q_out) + (n0 + x.t) * p.os + x.h * p.d;
            } else {
                const int64_t at = place[x.t].at;
                if (at < 0) return;
                const bool is_v = x.h >= p.Hq + p.Hk;
                const int h = x.h - p.Hq - (is_v ? p.Hk : 0);
                dst = reinterpret_cast<T *>(is_v ? p.v_pages : p.k_pages) + at + h * p.head_stride;
            }
            dst += offset(x.w);
            if (x.w < s.turned && (!APPEND || x.h < p.Hq + p.Hk)) {
                if constexpr (V == 1) {
                    const float2 c = angle2[x.t * half + x.w];
                    const float f1 = ld_f(&x.a.v[0]), f2 = ld_f(&x.b.v[0]);
                    x.a.v[0] = rounded<T>(fmaf(f1, c.x, -f2 * c.y));
                    x.b.v[0] = rounded<T>(fmaf(f2, c.x, f1 * c.y));
                } else {
                    const float4 *cs = angle4 + x.t * (half / 2) + x.w;
#pragma unroll
                    for (int q = 0; q < V / 2; ++q) {
                        const float4 c = cs[q * s.turned];
                        if constexpr (PAIRS) {  // a and b are 2 V elements in a row, a pair a word
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int j = 2 * q + e;
                                Vec<T, V> &y = j < V / 2 ? x.a : x.b;
                                const float2 f = get2(y, j % (V / 2));
                                const float cj = e ? c.y : c.x, sj = e ? c.w : c.z;
                                put2(y, j % (V / 2), __ffma2_rn(f, make_float2(cj, cj), __fmul2_rn(make_float2(f.y, f.x), make_float2(-sj, sj))));
                            }
                        } else {
                            const float2 f1 = get2(x.a, q), f2 = get2(x.b, q), c2 = make_float2(c.x, c.y);
                            put2(x.a, q, __ffma2_rn(f1, c2, __fmul2_rn(f2, make_float2(-c.z, -c.w))));
                            put2(x.b, q, __ffma2_rn(f2, c2, __fmul2_rn(f1, make_float2(c.z, c.w))));
                        }
                    }
                }
            }
            *reinterpret_cast<Vec<T, V> *>(dst) = x.a;
            if (x.w < s.turned) *reinterpret_cast<Vec<T, V> *>(dst + second) = x.b;
        };
        Item<T, V> x[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) load(threadIdx.x + u * kThreads, x[u]);
        __syncthreads();  // the last tokens' places and angles have been read
        if (APPEND) {
            for (int t = threadIdx.x / 32; t < tokens; t += kThreads / 32) {
                const Place at = place_of(p, n0 + t);
                if (threadIdx.x % 32 == 0) place[t] = at;
            }
            __syncthreads();
        }
        for (int e = threadIdx.x; e < tokens * half; e += kThreads) {
            const int t = (int)s.per_half.div(e), i = e - t * half;
            const int pos = APPEND && p.pos == nullptr ? place[t].pos : p.pos[axis[i] * p.N + n0 + t];
            // In units of 2^-32 turns: the nearest quarter, and no more than an eighth of a turn
            // from there, so that the 24 bits of fp32 hold the small angle to 2^-24 of itself.
            const uint32_t frac = (uint32_t)((turns[i] * (uint64_t)(int64_t)pos) >> 32);
            const uint32_t quarter = (frac + 0x20000000u) >> 30;
            float c0, s0;
            sincospif((float)(int32_t)(frac - (quarter << 30)) * 0x1p-31f, &s0, &c0);
            float c = quarter & 1 ? s0 : c0, sn = quarter & 1 ? c0 : s0;
            if (quarter == 1 || quarter == 2) c = -c;
            if ((quarter >= 2) != ((p.flags & GDN_ROTARY_INVERSE) != 0)) sn = -sn;
            if constexpr (V == 1) {
                angle2[e] = make_float2(c, sn);
            } else {
                const int w = i / V, j = i % V;
                float *at = reinterpret_cast<float *>(angle4 + t * (half / 2) + j / 2 * s.turned + w) + j % 2;
                at[0] = c;
                at[2] = sn;
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) finish(x[u]);
        for (uint32_t e0 = threadIdx.x + kInFlight * kThreads; e0 < items; e0 += kInFlight * kThreads) {
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) load(e0 + u * kThreads, x[u]);
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) finish(x[u]);
        }
    }
}

template <typename T, int V, bool PAIRS, bool APPEND>
cudaError_t launch_v(const RotaryParams &p, cudaStream_t stream) {
    const int turned = p.R / 2 / V, rest = (p.d - p.R) / V;
    const uint32_t per_head = (uint32_t)(turned + rest);
    const uint32_t heads = (uint32_t)(p.Hq + (APPEND ? 2 * p.Hk : 0));
    RotaryShape s{1, turned, Divisor(per_head * heads), Divisor(per_head), Divisor(p.R > 0 ? p.R / 2 : 1)};
    // tokens a turn of the CTA: enough for its vectors in flight, where there are enough
    // tokens for every CTA that runs at once
    const int64_t ctas = (int64_t)sm_count_of_current_device() * kCtas;
    int64_t t = (kThreads * kInFlight + per_head * heads - 1) / (per_head * heads);
    t = t < p.N / ctas ? t : p.N / ctas;
    if (p.R > 0) t = t < 2 * kMaxAngles / p.R ? t : 2 * kMaxAngles / p.R;
    s.tokens = (int)(t < 1 ? 1 : t > kMaxTokens ? kMaxTokens : t);
    const int64_t grid = (p.N + s.tokens - 1) / s.tokens;
    rotary_kernel<T, V, PAIRS, APPEND><<<(unsigned)(grid < ctas ? grid : ctas), kThreads,
                                         (size_t)s.tokens * (p.R / 2) * sizeof(float2), stream>>>(p, s);
    return cudaGetLastError();
}

template <typename T, int V>
cudaError_t launch_e(const RotaryParams &p, int v, cudaStream_t stream) {
    if constexpr (V > 1)
        if (v < V) return launch_e<T, V / 2>(p, v, stream);
    const bool pairs = (p.flags & GDN_ROTARY_PAIRS) != 0, append = p.Hk > 0;
    if (pairs) return append ? launch_v<T, V, true, true>(p, stream) : launch_v<T, V, true, false>(p, stream);
    return append ? launch_v<T, V, false, true>(p, stream) : launch_v<T, V, false, false>(p, stream);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams &p, cudaStream_t stream) {
    // The largest vector that divides widths, strides and addresses (in elements).
    const int e = p.dt == GDN_F32 ? 4 : 2;
    uint64_t all = (uint64_t)(p.R / 2) | (uint64_t)(p.d - p.R) | (uint64_t)p.d;
    auto rows = [&](const void *x, int64_t stride) {
        if (x != nullptr) all |= reinterpret_cast<uintptr_t>(x) / e | (uint64_t)stride;
    };
    rows(p.q, p.qs);
    rows(p.q_out, p.os);
    rows(p.k, p.ks);
    rows(p.v, p.vs);
    if (p.Hk > 0) {
        rows(p.k_pages, p.page_stride | p.slot_stride | p.head_stride);
        rows(p.v_pages, 0);
    }
    int v = 16 / e;
    while (v > 1 && (all & (uint64_t)(v - 1)) != 0) v /= 2;
    if (p.dt == GDN_F32) return launch_e<float, 4>(p, v, stream);
    return p.dt == GDN_F16 ? launch_e<__half, 8>(p, v, stream) : launch_e<__nv_bfloat16, 8>(p, v, stream);
}

}  // namespace gdn
