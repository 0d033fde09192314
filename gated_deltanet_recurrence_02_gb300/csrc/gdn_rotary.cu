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
// 2^-52 of the fraction's own rounding.  Its upper 32 bits go to sincospi as half turns.
//
// One pass: every element is read and written once, and bound by HBM.  A CTA takes a few
// tokens at a time: their angles' cosines and sines go to shared memory once for all
// heads, then each thread moves vectors of V elements (16 bytes where the alignment and
// the widths allow) of a pair's both halves, four of them in flight.
#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 4;
constexpr int kMaxTokens = 32;   // a CTA at a time
constexpr int kMaxAngles = 2048; // of them together

// n / d for any 32-bit n by a multiplication: T. Granlund and P. Montgomery, "Division by
// invariant integers using multiplication" (1994), figure 4.1.
struct Divisor {
    uint32_t m, s1, s2, d;
    explicit Divisor(uint32_t d_) : d(d_) {
        uint32_t l = 0;
        while (l < 32 && (1ull << l) < d) ++l;
        m = (uint32_t)((((1ull << l) - d) << 32) / d + 1);
        s1 = l < 1 ? l : 1;
        s2 = l < 1 ? 0 : l - 1;
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        const uint32_t t = __umulhi(m, n);
        return (t + ((n - t) >> s1)) >> s2;
    }
};

struct RotaryShape {
    int tokens;        // a CTA at a time
    int turned, rest;  // vectors of a head: that turn (both halves), that are copied
    Divisor per_token, per_head;
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

// Where a token's keys and values go, and the position that turns them where none is given.
struct Place {
    int64_t at;  // elements into the pages, or -1: nowhere
    int pos;     // in the cache
    int row;     // its row, or -1: none
};

__device__ Place place_of(const RotaryParams &p, int64_t n) {
    Place x{-1, 0, -1};
    int b, t, len;
    if (p.cu_seqlens == nullptr) {
        b = (int)(n / p.T);
        t = (int)(n - (int64_t)b * p.T);
        len = p.T;
    } else {
        int lo = 0, hi = p.B;  // the last row that starts at or before n
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.cu_seqlens[mid] <= n) lo = mid;
            else hi = mid;
        }
        b = lo;
        long tok0;
        row_range(p.cu_seqlens, b, (int)p.N, tok0, len);
        if (n < tok0 || n >= tok0 + len) return x;
        t = (int)(n - tok0);
    }
    x.row = b;
    const int64_t pos = (int64_t)p.kv_lens[b] - len + t;
    x.pos = (int)pos;
    if (pos < 0) return x;  // before the cache's first position: kept nowhere
    const int64_t page = pos / p.page_size;
    int id = -1;
    if (page < p.max_pages) id = p.page_table[(int64_t)b * p.max_pages + page];
    if (id < 0 || id >= p.num_pages) {
        atomicOr(p.err, (uint32_t)GDN_DEVERR_BAD_INDEX);
        return x;
    }
    x.at = id * p.page_stride + (pos - page * p.page_size) * p.slot_stride;
    return x;
}

template <typename T, int V, bool PAIRS, bool APPEND>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p, const RotaryShape s) {
    extern __shared__ float2 angle[];  // [tokens][R / 2] cosine, sine
    __shared__ uint64_t turns[kRotaryMaxWidth / 2];
    __shared__ int axis[kRotaryMaxWidth / 2];
    __shared__ Place place[kMaxTokens];
    const int half = p.R / 2;
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
        if (APPEND && threadIdx.x < tokens) place[threadIdx.x] = place_of(p, n0 + threadIdx.x);
        __syncthreads();
        for (int e = threadIdx.x; e < tokens * half; e += kThreads) {
            const int t = e / half, i = e - t * half;
            const int pos = APPEND && p.pos == nullptr ? place[t].pos : p.pos[axis[i] * p.N + n0 + t];
            const int32_t frac = (int32_t)((turns[i] * (uint64_t)(int64_t)pos) >> 32);
            float c, sn;
            sincospif((float)frac * 0x1p-31f, &sn, &c);
            angle[e] = make_float2(c, (p.flags & GDN_ROTARY_INVERSE) ? -sn : sn);
        }
        __syncthreads();
        const uint32_t items = (uint32_t)tokens * s.per_token.d;
        for (uint32_t e0 = threadIdx.x; e0 < items; e0 += kThreads * kInFlight) {
            Vec<T, V> a[kInFlight], b[kInFlight];
            T *dst[kInFlight];
            int from[kInFlight];  // the pair's first angle, -1: copied, -2: nothing here
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                const uint32_t e = e0 + u * kThreads;
                from[u] = -2;
                if (e >= items) continue;
                const uint32_t t = s.per_token.div(e), r = e - t * s.per_token.d;
                const uint32_t h = s.per_head.div(r), w = r - h * s.per_head.d;
                const int64_t n = n0 + t;
                const T *src;
                bool turned = (int)w < s.turned;
                if (!APPEND || (int)h < p.Hq) {
                    if (APPEND && place[t].row < 0) continue;
                    src = reinterpret_cast<const T *>(p.q) + n * p.qs + (int64_t)h * p.d;
                    dst[u] = reinterpret_cast<T *>(p.q_out) + n * p.os + (int64_t)h * p.d;
                } else {
                    if (place[t].at < 0) continue;
                    const bool is_v = (int)h >= p.Hq + p.Hk;
                    const int kh = (int)h - p.Hq - (is_v ? p.Hk : 0);
                    src = reinterpret_cast<const T *>(is_v ? p.v : p.k) + n * (is_v ? p.vs : p.ks) + (int64_t)kh * p.d;
                    dst[u] = reinterpret_cast<T *>(is_v ? p.v_pages : p.k_pages) + place[t].at + kh * p.head_stride;
                    if (is_v && turned) turned = false, from[u] = -3;  // copied, both halves
                }
                // offset of the vector in its head; of halves the second one lies half further
                const int i = turned || from[u] == -3 ? (PAIRS ? 2 * V * (int)w : V * (int)w)
                                                      : p.R + V * ((int)w - s.turned);
                src += i;
                dst[u] += i;
                a[u] = *reinterpret_cast<const Vec<T, V> *>(src);
                if (turned || from[u] == -3) b[u] = *reinterpret_cast<const Vec<T, V> *>(src + (PAIRS ? V : half));
                if (turned) from[u] = (int)t * half + V * (int)w;
                else if (from[u] != -3) from[u] = -1;
            }
#pragma unroll
            for (int u = 0; u < kInFlight; ++u) {
                if (from[u] == -2) continue;
                if (from[u] >= 0) {
                    const float2 *cs = angle + from[u];
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        if constexpr (PAIRS) {  // (a, b) are 2 V elements in a row
                            T &x1 = 2 * j < V ? a[u].v[(2 * j) % V] : b[u].v[(2 * j) % V];
                            T &x2 = 2 * j + 1 < V ? a[u].v[(2 * j + 1) % V] : b[u].v[(2 * j + 1) % V];
                            const float f1 = ld_f(&x1), f2 = ld_f(&x2);
                            x1 = rounded<T>(fmaf(f1, cs[j].x, -f2 * cs[j].y));
                            x2 = rounded<T>(fmaf(f2, cs[j].x, f1 * cs[j].y));
                        } else {
                            const float f1 = ld_f(&a[u].v[j]), f2 = ld_f(&b[u].v[j]);
                            a[u].v[j] = rounded<T>(fmaf(f1, cs[j].x, -f2 * cs[j].y));
                            b[u].v[j] = rounded<T>(fmaf(f2, cs[j].x, f1 * cs[j].y));
                        }
                    }
                }
                *reinterpret_cast<Vec<T, V> *>(dst[u]) = a[u];
                if (from[u] != -1) *reinterpret_cast<Vec<T, V> *>(dst[u] + (PAIRS ? V : half)) = b[u];
            }
        }
        __syncthreads();
    }
}

template <typename T, int V, bool PAIRS, bool APPEND>
cudaError_t launch_v(const RotaryParams &p, cudaStream_t stream) {
    const int turned = p.R / 2 / V, rest = (p.d - p.R) / V;
    const uint32_t per_head = (uint32_t)(turned + rest);
    const uint32_t heads = (uint32_t)(p.Hq + (APPEND ? 2 * p.Hk : 0));
    RotaryShape s{1, turned, rest, Divisor(per_head * heads), Divisor(per_head)};
    // tokens a turn of the CTA: enough for its vectors in flight, where there are enough
    // tokens for every CTA that runs at once
    const int64_t ctas = (int64_t)sm_count_of_current_device() * (2048 / kThreads);
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
