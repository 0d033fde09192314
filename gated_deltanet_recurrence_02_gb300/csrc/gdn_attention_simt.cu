// gdn_attention_simt.cu -- attention over a paged cache on the CUDA cores: fp32, and 16-bit
// tensors whose strides or page size the tensor-core kernel does not take.  Also the join of
// both kernels' cut units and the choice between them.
//
// Per query row, over tiles of keys, with running maximum m and sum l (both of scores times
// scale log2 e, so that weights are powers of two):
//     x_j = scale log2 e q.k_j,  m' = max(m, max_j x_j),  w_j = 2^{x_j - m'}
//     l <- 2^{m - m'} l + sum_j w_j,   o <- 2^{m - m'} o + sum_j w_j v_j
// and o / l at the end; all in fp32.  A key that a query does not see gets no weight and its
// values are not added, whatever they hold.  A row without keys gives 0 and a log of -inf.
//
// A CTA of 64 (or, for few rows, 16) query rows holds them, a tile of keys and one of values
// in shared memory; a thread has four rows of a few keys, then of a few output features.
#include <algorithm>

#include "gdn_attention.cuh"

namespace gdn {
namespace attn {
namespace {

template <int M>
struct Shape {
    static constexpr int TX = M == 64 ? 16 : 32;       // threads along keys and features
    static constexpr int kThreads = M / 4 * TX;
    static constexpr int KT = M == 64 ? 32 : 64;       // keys of a tile
};

template <typename T, int D, int M>
__global__ void __launch_bounds__(Shape<M>::kThreads) simt_kernel(const AttentionParams p, const Plan s, bool vectors) {
    constexpr int TX = Shape<M>::TX, KT = Shape<M>::KT, THREADS = Shape<M>::kThreads;
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
                if (vectors) x = ld4(g + c);
                else x = make_float4(ld_f(g + c), ld_f(g + c + 1), ld_f(g + c + 2), ld_f(g + c + 3));
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
            lo[i] = p.causal && p.window > 0 ? max(0, at - p.window + 1) : 0;
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

template <typename T, int D, int M>
cudaError_t launch_m(const AttentionParams &p, const Plan &s, cudaStream_t stream) {
    using S = Shape<M>;
    constexpr int bytes = (M * D + S::KT * (2 * D + 4) + M * (S::KT + 4)) * (int)sizeof(float);
    cudaError_t e = set_smem_once<simt_kernel<T, D, M>>(bytes);
    if (e != cudaSuccess) return e;
    const uintptr_t all = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k_pages) |
                          reinterpret_cast<uintptr_t>(p.v_pages) |
                          (uintptr_t)(p.qs | p.page_stride | p.slot_stride | p.head_stride) * sizeof(T);
    simt_kernel<T, D, M><<<s.ctas, S::kThreads, bytes, stream>>>(p, s, (all & (4 * sizeof(T) - 1)) == 0);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join(p, s, stream);
}

template <typename T>
cudaError_t launch_t(const AttentionParams &p, const Plan &s, cudaStream_t stream) {
    const bool few = s.rows() <= 16;
    switch (p.d) {
        case 32: return few ? launch_m<T, 32, 16>(p, s, stream) : launch_m<T, 32, 64>(p, s, stream);
        case 64: return few ? launch_m<T, 64, 16>(p, s, stream) : launch_m<T, 64, 64>(p, s, stream);
        default: return few ? launch_m<T, 128, 16>(p, s, stream) : launch_m<T, 128, 64>(p, s, stream);
    }
}

template <typename T, int D>
cudaError_t launch_join_d(const AttentionParams &p, const Plan &s, cudaStream_t stream) {
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
    const cudaError_t e = cudaLaunchKernelEx(&cfg, join_kernel<T, D>, p, s);
    return e != cudaSuccess ? e : cudaGetLastError();
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

// Query rows a unit: 16 where a row of the batch has no more on average, else 64.
Plan plan_simt(int B, int T, int Hq, int Hk, int d, bool varlen) {
    const int rows = mean_tokens(B, T, varlen) * (Hq / Hk) <= 16 ? 16 : 64;
    return plan_of(Hq, Hk, d, rows, 2 * sm_count_of_current_device(), 1, 1);
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
