// gdn_attention_simt.cu -- attention over a paged cache on the CUDA cores: fp32, and 16-bit
// tensors whose addresses or strides are no multiples of 16 bytes.  Also the join of both
// kernels' cut units and the choice between them.
//
// Per query row, over tiles of keys, with running maximum m and sum l (both of scores times
// scale log2 e, so that weights are powers of two):
//     x_j = scale log2 e q.k_j,  m' = max(m, max_j x_j),  w_j = 2^{x_j - m'}
//     l <- 2^{m - m'} l + sum_j w_j,   o <- 2^{m - m'} o + sum_j w_j v_j
// and o / l at the end; all in fp32.  A key that a query does not see gets no weight and its
// values are not added, whatever they hold.  A row without keys gives 0 and a log of -inf; a
// score that is NaN makes its row NaN.
//
// Two kernels.  Of up to 8 query rows (single tokens, a few drafts): a warp streams keys and
// values through registers, four features a lane, and has all rows' queries and sums in
// registers too.  Of up to 4 rows bound by HBM, single tokens of 64 rows over 2000 keys, 4 of
// 16 heads, d = 128, fp32: 105 us, 5.0 TB/s; of 8 by the sums over the lanes, 159 us for the
// same bytes.  Of up to 64: a CTA holds them, a tile of keys and one of values in shared
// memory, bound by the shared memory that feeds the FMA units (six 16-byte loads for 32 FMAs);
// a thread has four rows of a few keys, then of a few output features.  4 x 1000 tokens over
// 2000 keys each, the same heads: 1.69 ms, 39 TFLOP/s.
#include <algorithm>

#include "gdn_attention.cuh"

namespace gdn {
namespace attn {
namespace {

constexpr int kLanes = 16;        // threads along keys and features
constexpr int kThreads = 256;
constexpr int kRows = 64, kKeys = 32;  // query rows, keys of a tile
constexpr int kStreamKeys = 64;   // of a tile, where keys are streamed

// Four elements of a row in fp32; `vectors`: 16 (or, of 16 bits, 8) bytes aligned.
template <typename T>
__device__ __forceinline__ float4 load4(const T *g, bool vectors) {
    if (vectors) return ld4(g);
    return make_float4(ld_f(g), ld_f(g + 1), ld_f(g + 2), ld_f(g + 3));
}

// Up to R query rows.  A key takes D / 4 lanes, so a warp has K = 128 / D keys at a time and
// U times as many on their way; the warps of a CTA take the piece's keys in turn.  Each group
// of lanes has sums and maxima of its own, joined at the unit's end through shared memory.
template <typename T, int D, int R>
__global__ void __launch_bounds__(kThreads, 2) stream_kernel(const AttentionParams p, const Plan s,
                                                              const Divisor page_size, bool vectors) {
    constexpr int L = D / 4, K = 32 / L, U = R == 4 ? 4 : 2, kWarps = kThreads / 32, kGroups = kWarps * K;
    static_assert(R <= L, "the scores of one row end up in a lane");
    extern __shared__ float4 smem4[];
    float4 *parts = smem4;                                                       // [kGroups][R][L]
    float2 *part_stats = reinterpret_cast<float2 *>(smem4 + kGroups * R * L);    // [kGroups][R]
    const Place from = find_place<kStreamKeys, kThreads>(p, s);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, in = lane % L, sub = lane / L;
    const float scale2 = p.scale * tc::kLog2e;
    // The lane's row (others of the group may have the same): row bits from the top are lane
    // bits from the top of the group's.
    int own = 0;
#pragma unroll
    for (int n = R, o = L / 2; n > 1 && o > 0; n /= 2, o /= 2) own += in & o ? n / 2 : 0;
    auto owner = [](int r) {  // a lane of the group that has row r
        int x = 0;
#pragma unroll
        for (int n = R, o = L / 2; n > 1 && o > 0; n /= 2, o /= 2) {
            if (r >= n / 2) x += o, r -= n / 2;
        }
        return x;
    };
    Walk<kStreamKeys> w;
    Cut cut{};
    for (bool more = w.start(p, s, from); more; more = w.next(p, s)) {
        const Unit &u = w.unit;
        const int n = u.t1 - u.t0, heads = w.heads(p, s), head0 = w.head0(p, s), hk = w.key_head(s);
        cut = w.cut(p, s);
        float4 q[R], acc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int t = r / s.gs, g = r - t * s.gs;
            q[r] = acc[r] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t < n && g < heads) {
                q[r] = load4(reinterpret_cast<const T *>(p.q) + (w.row.tok0 + u.t0 + t) * p.qs + (int64_t)(head0 + g) * D + 4 * in,
                             vectors);
                q[r] = make_float4(q[r].x * scale2, q[r].y * scale2, q[r].z * scale2, q[r].w * scale2);
            }
        }
        float m = kNone, l = 0.f;
        int lo, hi;                           // keys that the lane's row sees
        int all_lo = 0, all_hi = 0x7fffffff;  // that all of them see
        auto sees = [&](int r, int &a, int &b) {
            const int at = w.row.first + u.t0 + min(r / s.gs, n - 1);
            a = window_start(p, at);
            b = p.causal ? min(w.row.keys, at + 1) : w.row.keys;
        };
        sees(own, lo, hi);
        {
            int a, b;
            sees((n - 1) * s.gs, all_lo, b);
            sees(0, a, all_hi);
        }
        const int k1 = min(u.hi, u.key0 + w.end * kStreamKeys);
        int k0 = max(u.lo, u.key0 + w.at.tile * kStreamKeys) + warp * (K * U);
        const int32_t *table = p.page_table + (int64_t)w.at.b * p.max_pages;
        // Pages of the group's next keys, read a turn ahead
        int page[U];
        auto pages_of = [&](int k) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int key = k + j * K + sub;
                page[j] = key < k1 ? table[page_size.div((uint32_t)key)] : -1;
            }
        };
        pages_of(k0);
        for (; k0 < k1; k0 += kWarps * K * U) {
            float4 kk[U], vv[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int key = k0 + j * K + sub, id = page[j];
                kk[j] = vv[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (id >= 0 && id < p.num_pages) {
                    const uint32_t slot = (uint32_t)key - page_size.div((uint32_t)key) * page_size.d;
                    const int64_t at = id * p.page_stride + (int64_t)slot * p.slot_stride + hk * p.head_stride + 4 * in;
                    kk[j] = load4(reinterpret_cast<const T *>(p.k_pages) + at, vectors);
                    vv[j] = load4(reinterpret_cast<const T *>(p.v_pages) + at, vectors);
                } else if (key < k1) {
                    atomicOr(p.err, (uint32_t)GDN_DEVERR_BAD_INDEX);
                }
            }
            pages_of(k0 + kWarps * K * U);
            float x[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                float v[R];
#pragma unroll
                for (int r = 0; r < R; ++r)
                    v[r] = fmaf(q[r].x, kk[j].x, fmaf(q[r].y, kk[j].y, fmaf(q[r].z, kk[j].z, q[r].w * kk[j].w)));
                // Sums over the group's lanes, in each step of half as many rows
                int rows = R;
#pragma unroll
                for (int o = L / 2; o > 0; o /= 2) {
                    if (rows > 1) {
                        rows /= 2;
                        const bool up = (in & o) != 0;
#pragma unroll
                        for (int r = 0; r < R / 2; ++r) {
                            if (r >= rows) break;
                            const float got = __shfl_xor_sync(kAll, up ? v[r] : v[r + rows], o);
                            v[r] = (up ? v[r + rows] : v[r]) + got;
                        }
                    } else {
                        v[0] += __shfl_xor_sync(kAll, v[0], o);
                    }
                }
                const int key = k0 + j * K + sub;
                x[j] = key < k1 && key >= lo && key < hi ? v[0] : kNone;
            }
            // (the maximum that weights are relative to follows the true one when that has grown
            // by more than 8 in the exponent, as in the tensor-core kernel)
            float now = m;
#pragma unroll
            for (int j = 0; j < U; ++j) now = fmaxf(now, x[j]);
            if (__any_sync(kAll, now - m > 8.f)) {
                const float keep = now == kNone ? 1.f : exp2f(m - now);
                m = now;
                l *= keep;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float f = __shfl_sync(kAll, keep, sub * L + owner(r));
                    acc[r] = make_float4(acc[r].x * f, acc[r].y * f, acc[r].z * f, acc[r].w * f);
                }
            }
            // (no maximum yet: every key so far is hidden, x = -infinity and no weight, or NaN, which
            // a maximum passes over and the weight keeps)
            const float safe = m == kNone ? 0.f : m;
            const bool tested = k0 < all_lo || k0 + K * U > all_hi;  // a row may not see a key
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const float e = exp2f(x[j] - safe);
                l += e;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const float f = __shfl_sync(kAll, e, sub * L + owner(r));
                    if (tested && f == 0.f) continue;  // (what a hidden key's values are does not matter)
                    acc[r] = make_float4(fmaf(f, vv[j].x, acc[r].x), fmaf(f, vv[j].y, acc[r].y),
                                         fmaf(f, vv[j].z, acc[r].z), fmaf(f, vv[j].w, acc[r].w));
                }
            }
        }
        __syncthreads();  // the last unit's parts have been read
        const int group = warp * K + sub;
#pragma unroll
        for (int r = 0; r < R; ++r) parts[(group * R + r) * L + in] = acc[r];
        part_stats[group * R + own] = make_float2(m, l);
        __syncthreads();
        for (int e = threadIdx.x; e < R * L; e += kThreads) {
            const int r = e / L, c = e % L, t = r / s.gs, g = r - t * s.gs;
            if (t >= n || g >= heads) continue;
            float top = kNone;
            for (int y = 0; y < kGroups; ++y) top = fmaxf(top, part_stats[y * R + r].x);
            const float safe = top == kNone ? 0.f : top;
            float sum = 0.f;
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int y = 0; y < kGroups; ++y) {
                const float2 ml = part_stats[y * R + r];
                const float4 v = parts[(y * R + r) * L + c];
                const float f = exp2f(ml.x - safe);
                sum = fmaf(f, ml.y, sum);
                a = make_float4(fmaf(f, v.x, a.x), fmaf(f, v.y, a.y), fmaf(f, v.z, a.z), fmaf(f, v.w, a.w));
            }
            if (w.part() < 0) {
                const long at = (w.row.tok0 + u.t0 + t) * p.Hq + head0 + g;
                const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;  // (a NaN stays one)
                T *out = reinterpret_cast<T *>(p.out) + at * D + 4 * c;
                st_out(out, a.x * inv);
                st_out(out + 1, a.y * inv);
                st_out(out + 2, a.z * inv);
                st_out(out + 3, a.w * inv);
                if (p.lse != nullptr && c == 0) p.lse[at] = (safe + log2f(sum)) * 0.69314718055994530942f;
            } else {
                *reinterpret_cast<float4 *>(s.sums(blockIdx.x, w.part()) + (size_t)r * D + 4 * c) = a;
                if (c == 0) s.stats(blockIdx.x, w.part())[r] = make_float2(top, sum);
            }
        }
    }
    if (threadIdx.x == 0) *s.cut(blockIdx.x) = cut;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) simt_kernel(const AttentionParams p, const Plan s, bool vectors) {
    constexpr int TX = kLanes, KT = kKeys, THREADS = kThreads, M = kRows;
    constexpr int NK = KT / TX, NC = D / TX, VC = NC < 4 ? NC : 4;
    extern __shared__ float4 smem4[];
    float *sq = reinterpret_cast<float *>(smem4);  // [M][D]
    float *sk = sq + M * D;                        // [KT][D + 4]
    float *sv = sk + KT * (D + 4);                 // [KT][D]
    float *sp = sv + KT * D;                       // [M][KT + 4]
    const int tx = threadIdx.x % TX, ty = threadIdx.x / TX;
    const Place from = find_place<KT, THREADS>(p, s);
    int tt[4], gg[4];  // token and head of the thread's rows in the unit
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        tt[i] = (ty * 4 + i) / s.gs;
        gg[i] = ty * 4 + i - tt[i] * s.gs;
    }
    const float scale2 = p.scale * tc::kLog2e;
    // Rows of D elements from global to shared memory as fp32; src(row) is the address or
    // nullptr (zeros).
    auto fill = [&](float *dst, int stride, int rows, auto src) {
        constexpr int VEC = 4;
        for (int e = threadIdx.x; e < rows * (D / VEC); e += THREADS) {
            const int r = e / (D / VEC), c = e % (D / VEC) * VEC;
            const T *g = src(r);
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (g != nullptr) {
                x = load4(g + c, vectors);
            }
            *reinterpret_cast<float4 *>(dst + r * stride + c) = x;
        }
    };
    Walk<KT> w;
    Cut cut{};
    for (bool more = w.start(p, s, from); more; more = w.next(p, s)) {
        const Unit &u = w.unit;
        const int n = u.t1 - u.t0, heads = w.heads(p, s), head0 = w.head0(p, s), hk = w.key_head(s);
        cut = w.cut(p, s);
        __syncthreads();
        fill(sq, D, M, [&](int r) -> const T * {
            const int t = r / s.gs, g = r - t * s.gs;
            if (t >= n || g >= heads) return nullptr;
            return reinterpret_cast<const T *>(p.q) + (w.row.tok0 + u.t0 + t) * p.qs + (int64_t)(head0 + g) * D;
        });
        float m[4], l[4], o[4][NC];
        int lo[4], hi[4];  // keys that a row sees
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = kNone;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) o[i][c] = 0.f;
            const int at = w.row.first + u.t0 + min(tt[i], n - 1);
            lo[i] = window_start(p, at);
            hi[i] = p.causal ? min(w.row.keys, at + 1) : w.row.keys;
        }
        for (int tile = w.at.tile; tile < w.end; ++tile) {
            const int k0 = u.key0 + tile * KT;
            __syncthreads();
            auto page = [&](const void *pages) {
                return [&, pages](int r) -> const T * {
                    const int k = k0 + r;
                    if (k < u.lo || k >= u.hi) return nullptr;
                    const int pg = k / p.page_size;
                    const int id = p.page_table[(int64_t)w.at.b * p.max_pages + pg];
                    if (id < 0 || id >= p.num_pages) {
                        atomicOr(p.err, (uint32_t)GDN_DEVERR_BAD_INDEX);
                        return nullptr;
                    }
                    return reinterpret_cast<const T *>(pages) + id * p.page_stride +
                           (int64_t)(k - pg * p.page_size) * p.slot_stride + hk * p.head_stride;
                };
            };
            fill(sk, D + 4, KT, page(p.k_pages));
            fill(sv, D, KT, page(p.v_pages));
            __syncthreads();
            float x[4][NK];
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < NK; ++j) x[i][j] = 0.f;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                float4 q[4], k[NK];
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const float4 *>(sq + (ty * 4 + i) * D + c);
#pragma unroll
                for (int j = 0; j < NK; ++j) k[j] = *reinterpret_cast<const float4 *>(sk + (tx + TX * j) * (D + 4) + c);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < NK; ++j) {
                        x[i][j] = fmaf(q[i].x, k[j].x, x[i][j]);
                        x[i][j] = fmaf(q[i].y, k[j].y, x[i][j]);
                        x[i][j] = fmaf(q[i].z, k[j].z, x[i][j]);
                        x[i][j] = fmaf(q[i].w, k[j].w, x[i][j]);
                    }
            }
            bool hidden = false;  // a key of the tile is hidden from one of the thread's rows
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float top = m[i];
#pragma unroll
                for (int j = 0; j < NK; ++j) {
                    const int k = k0 + tx + TX * j;
                    const bool see = k >= lo[i] && k < hi[i];
                    x[i][j] = see ? x[i][j] * scale2 : kNone;
                    top = fmaxf(top, x[i][j]);
                }
                hidden |= k0 < lo[i] || k0 + KT > hi[i];
#pragma unroll
                for (int d = TX / 2; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
                const float safe = top == kNone ? 0.f : top, keep = exp2f(m[i] - safe);
                float sum = 0.f;
#pragma unroll
                for (int j = 0; j < NK; ++j) {
                    const float e = exp2f(x[i][j] - safe);
                    sum += e;
                    sp[(ty * 4 + i) * (KT + 4) + tx + TX * j] = e;
                }
                l[i] = fmaf(l[i], keep, sum);  // (this thread's keys; added up at the end)
                m[i] = top;
#pragma unroll
                for (int c = 0; c < NC; ++c) o[i][c] *= keep;
            }
            __syncwarp();
            // (in two copies: only a tile with hidden keys tests each key)
            auto add = [&](auto tested) {
#pragma unroll 2
                for (int k = 0; k < KT; k += 4) {
                    float4 e4[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) e4[i] = *reinterpret_cast<const float4 *>(sp + (ty * 4 + i) * (KT + 4) + k);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        float v[NC];
#pragma unroll
                        for (int c = 0; c < NC; c += VC)
#pragma unroll
                            for (int e = 0; e < VC; ++e) v[c + e] = sv[(k + kk) * D + (c / VC) * TX * VC + tx * VC + e];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float e = kk == 0 ? e4[i].x : kk == 1 ? e4[i].y : kk == 2 ? e4[i].z : e4[i].w;
                            if (decltype(tested)::value && !(k0 + k + kk >= lo[i] && k0 + k + kk < hi[i])) continue;
#pragma unroll
                            for (int c = 0; c < NC; ++c) o[i][c] = fmaf(e, v[c], o[i][c]);
                        }
                    }
                }
            };
            if (__any_sync(0xffffffffu, hidden)) add(std::true_type{});
            else add(std::false_type{});
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int d = TX / 2; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
            const int r = ty * 4 + i;
            if (tt[i] >= n || gg[i] >= heads) continue;
            if (w.part() < 0) {
                const long at = (w.row.tok0 + u.t0 + tt[i]) * p.Hq + head0 + gg[i];
                const float inv = l[i] > 0.f ? 1.f / l[i] : l[i] == 0.f ? 0.f : l[i];  // (a NaN stays one)
                T *out = reinterpret_cast<T *>(p.out) + at * D;
#pragma unroll
                for (int c = 0; c < NC; ++c) st_out(out + (c / VC) * TX * VC + tx * VC + c % VC, o[i][c] * inv);
                if (p.lse != nullptr && tx == 0)
                    p.lse[at] = ((m[i] == kNone ? 0.f : m[i]) + log2f(l[i])) * 0.69314718055994530942f;
            } else {
                float *out = s.sums(blockIdx.x, w.part()) + (size_t)r * D;
#pragma unroll
                for (int c = 0; c < NC; ++c) out[(c / VC) * TX * VC + tx * VC + c % VC] = o[i][c];
                if (tx == 0) s.stats(blockIdx.x, w.part())[r] = make_float2(m[i], l[i]);
            }
        }
    }
    if (threadIdx.x == 0) *s.cut(blockIdx.x) = cut;
}

template <typename T, int D, int R>
cudaError_t launch_stream(const AttentionParams &p, const Plan &s, bool vectors, cudaStream_t stream) {
    constexpr int bytes = kThreads / 32 * (R * 128 * (int)sizeof(float) + 128 / D * R * (int)sizeof(float2));
    cudaError_t e = set_smem_once<stream_kernel<T, D, R>>(bytes);
    if (e != cudaSuccess) return e;
    stream_kernel<T, D, R><<<s.ctas, kThreads, bytes, stream>>>(p, s, Divisor((uint32_t)p.page_size), vectors);
    return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_d(const AttentionParams &p, const Plan &s, cudaStream_t stream) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k_pages) |
                          reinterpret_cast<uintptr_t>(p.v_pages) |
                          (uintptr_t)(p.qs | p.page_stride | p.slot_stride | p.head_stride) * sizeof(T);
    const bool vectors = (all & (4 * sizeof(T) - 1)) == 0;
    cudaError_t e;
    if (s.rows() <= 4) {
        e = launch_stream<T, D, 4>(p, s, vectors, stream);
    } else if (s.rows() <= 8) {
        e = launch_stream<T, D, 8>(p, s, vectors, stream);
    } else {
        constexpr int bytes = (kRows * D + kKeys * (2 * D + 4) + kRows * (kKeys + 4)) * (int)sizeof(float);
        e = set_smem_once<simt_kernel<T, D>>(bytes);
        if (e != cudaSuccess) return e;
        simt_kernel<T, D><<<s.ctas, kThreads, bytes, stream>>>(p, s, vectors);
        e = cudaGetLastError();
    }
    return e != cudaSuccess ? e : launch_join(p, s, stream);
}

template <typename T>
cudaError_t launch_t(const AttentionParams &p, const Plan &s, cudaStream_t stream) {
    switch (p.d) {
        case 32: return launch_d<T, 32>(p, s, stream);
        case 64: return launch_d<T, 64>(p, s, stream);
        default: return launch_d<T, 128>(p, s, stream);
    }
}

template <typename T, int D, bool SHARE>
cudaError_t launch_join_s(const AttentionParams &p, const Plan &s, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    // (a warp has four rows at a time, a CTA eight warps; no more CTAs than run at once)
    const long most = std::min<long>(s.rows(), (long)p.T * s.gs);  // query rows of a unit
    cfg.gridDim = dim3((unsigned)s.ctas, (unsigned)std::min<long>((most + 31) / 32, 4));
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, join_kernel<T, D, SHARE>, p, s);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_join_d(const AttentionParams &p, const Plan &s, cudaStream_t stream) {
    return mean_tokens(p.B, p.T, p.cu_seqlens != nullptr) * s.gs <= 16 ? launch_join_s<T, D, true>(p, s, stream)
                                                                       : launch_join_s<T, D, false>(p, s, stream);
}

template <typename T>
cudaError_t launch_join_t(const AttentionParams &p, const Plan &s, cudaStream_t stream) {
    switch (p.d) {
        case 32: return launch_join_d<T, 32>(p, s, stream);
        case 64: return launch_join_d<T, 64>(p, s, stream);
        default: return launch_join_d<T, 128>(p, s, stream);
    }
}

}  // namespace

cudaError_t launch_join(const AttentionParams &p, const Plan &s, cudaStream_t stream) {
    if (p.dt == GDN_F32) return launch_join_t<float>(p, s, stream);
    return p.dt == GDN_F16 ? launch_join_t<__half>(p, s, stream) : launch_join_t<__nv_bfloat16>(p, s, stream);
}

cudaError_t launch_attention_simt(const AttentionParams &p, const Plan &s, cudaStream_t stream) {
    if (p.dt == GDN_F32) return launch_t<float>(p, s, stream);
    return p.dt == GDN_F16 ? launch_t<__half>(p, s, stream) : launch_t<__nv_bfloat16>(p, s, stream);
}

// Query rows a unit.  Four are streamed at the rate of their bytes, eight at half of it (the
// sums over the lanes), so eight are the better from five rows on, and 64 by the other kernel
// once the rows of a key head fill six units of eight.  64 rows of the batch over 2000 keys,
// 4 key heads, d = 128, fp32, us by units of 4, 8, 64: of 4 query rows 106, 156, 679; of 8
// 198, 159, 680; of 20 469, 434, 677; of 32 742, 574, 682.  At 40 rows 8 and 64 meet (d = 128:
// 351 and 354, d = 64: 193 and 194), at 48 they are 438 and 355.  (16 rows a unit took what two
// units of 8 take.)
Plan plan_simt(int B, int T, int Hq, int Hk, int d, bool varlen) {
    const long rows = mean_tokens(B, T, varlen) * (Hq / Hk);
    return plan_of(Hq, Hk, d, rows <= 4 ? 4 : rows <= 40 ? 8 : kRows, 2 * sm_count_of_current_device(), 1, 1);
}

}  // namespace attn

// (for either kernel: strides and pages, which decide, are not among the sizes)
size_t attention_workspace_bytes(int B, int T, int Hq, int Hk, int d, int dt, bool varlen) {
    const size_t simt = attn::plan_simt(B, T, Hq, Hk, d, varlen).bytes();
    return dt == GDN_F32 ? simt : std::max(simt, attn::plan_tc(B, T, Hq, Hk, d, varlen).bytes());
}

cudaError_t launch_attention(const AttentionParams &p, cudaStream_t stream) {
    const bool varlen = p.cu_seqlens != nullptr, tc = attn::tc_takes(p);
    attn::Plan s = tc ? attn::plan_tc(p.B, p.T, p.Hq, p.Hk, p.d, varlen) : attn::plan_simt(p.B, p.T, p.Hq, p.Hk, p.d, varlen);
    s.ws = static_cast<uint8_t *>(p.ws);
    return tc ? attn::launch_attention_tc(p, s, stream) : attn::launch_attention_simt(p, s, stream);
}

}  // namespace gdn
