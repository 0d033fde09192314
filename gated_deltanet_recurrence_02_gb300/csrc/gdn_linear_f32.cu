// gdn_linear_f32.cu -- linear attention with a decay for each head over prompts,
// for fp32 inputs: S <- alpha S + v k^T, o = S (scale q), token by token on the
// CUDA cores, so every product and sum is fp32 and no decay is ever divided out.
//
// One CTA (128 threads) holds 16 R rows (value features) of one (row, value head)
// state in registers: each lane dk/8 columns of R rows as fp32 pairs.  Tokens
// come to shared memory kTokens at a time by cp.async, two blocks ahead; a block
// is then worked through without a barrier.  The readout's sums over the eight
// lanes of a row are taken for four tokens at once (a reduce-scatter of 4 R = 16
// values costs 14 shuffles, sixteen separate butterflies 48).
//
// Bound by fp32 arithmetic: 3 dk dv multiplications and fused multiply-adds a token and
// head (the decayed state, the update, the readout), 172 us for 4100 tokens of 32 heads
// with dk = dv = 128 on all SMs and two thirds of that again for the segments' first
// pass, against 30 us of HBM time.  Measured there: 431 us (four state rows a lane;
// 554 us with two, which loads k and q twice as often from shared memory).  The chunked
// form on the tensor cores would need each operand as sums of tf32 numbers and three
// products for each (about 40 us of tensor time at that size): not built; 16-bit inputs
// are the ones that prompts come in.
//
// Few rows are cut into segments, as on the tensor-core path: a first pass forms
// each segment's end state from zeros (the first one from the initial state), the
// second takes each segment's start from those.
#include "gdn_internal.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kTokens = 16;  // a block
constexpr int kBlocks = 3;   // blocks in shared memory

struct F32Params : PrefillParams {
    int G, G_run;
    float *seg_state, *seg_decay;
};

template <int DK, int R>
struct Block {
    float k[kTokens][DK], q[kTokens][DK], v[kTokens][16 * R], alpha[kTokens];
};

__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src)
                 : "memory");
}

// R: rows a lane; a CTA holds 16 R.
template <int DK, int R, bool kStateOnly>
__global__ void __launch_bounds__(kThreads) linear_f32_kernel(const F32Params p) {
    constexpr int F2 = DK / 16;  // pairs of a lane's columns of one row
    constexpr int kRows = 16 * R;
    extern __shared__ float4 smem4[];
    Block<DK, R> *blocks = reinterpret_cast<Block<DK, R> *>(smem4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = lane >> 3, l8 = lane & 7;
    const int Hv = p.Hv, Hk = p.Hk, dv = p.dv;
    const int tiles = dv / kRows;
    unsigned u = blockIdx.x;
    const int tile = (int)(u % tiles);
    u /= tiles;
    const int h = (int)(u % Hv);
    u /= Hv;
    const int g = (int)(u % p.G_run), b = (int)(u / p.G_run);
    const int hk = h / (Hv / Hk);
    long tok0;
    int len;
    row_range(p.cu_seqlens, b, p.T, tok0, len);
    const int per = ((len + p.G - 1) / p.G + kTokens - 1) / kTokens * kTokens;
    const int t_lo = min((int)min((long)g * per, (long)len), len), t_hi = min(t_lo + per, len);

    // the lane's R rows (of the state and of v) from row0 on, and columns 4 (f 8 + l8) + ..
    const int row0 = (warp * 4 + grp) * R;
    float2 S[R][F2];
    const size_t mat = (size_t)dv * DK, seg0 = ((size_t)b * Hv + h) * p.G;
    auto add_rows = [&](const float *m, float keep) {  // S <- keep S + the matrix's rows
        const float2 k2 = make_float2(keep, keep);
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int f = 0; f < F2 / 2; ++f) {
                const float4 x =
                    *reinterpret_cast<const float4 *>(m + (size_t)(tile * kRows + row0 + r) * DK + (f * 8 + l8) * 4);
                S[r][2 * f] = __ffma2_rn(k2, S[r][2 * f], make_float2(x.x, x.y));
                S[r][2 * f + 1] = __ffma2_rn(k2, S[r][2 * f + 1], make_float2(x.z, x.w));
            }
    };
    auto store_rows = [&](float *m) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int f = 0; f < F2 / 2; ++f)
                __stcs(reinterpret_cast<float4 *>(m + (size_t)(tile * kRows + row0 + r) * DK + (f * 8 + l8) * 4),
                       make_float4(S[r][2 * f].x, S[r][2 * f].y, S[r][2 * f + 1].x, S[r][2 * f + 1].y));
    };
    auto clear = [&]() {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int f = 0; f < F2; ++f) S[r][f] = make_float2(0.f, 0.f);
    };

    const float *kb = reinterpret_cast<const float *>(p.k) + (tok0 * Hk + hk) * DK;
    const float *qb = reinterpret_cast<const float *>(p.q) + (tok0 * Hk + hk) * DK;
    const float *vb = reinterpret_cast<const float *>(p.v) + (tok0 * Hv + h) * (long)dv + tile * kRows;
    float *ob = reinterpret_cast<float *>(p.out) + (tok0 * Hv + h) * (long)dv + tile * kRows;
    const long k_step = (long)Hk * DK, v_step = (long)Hv * dv;
    const int n_blocks = (t_hi - t_lo + kTokens - 1) / kTokens;
    float a_next = 1.f;  // decay of token tid of the next block
    auto fetch_alpha = [&](int blk) {
        const int t = t_lo + blk * kTokens + tid;
        if (tid < kTokens && t < t_hi)
            a_next = conv_alpha(ld_gate(p.alpha, (p.conv & GDN_ALPHA_PER_HEAD) ? h : (tok0 + t) * Hv + h, p.dt_gate), p.conv);
    };
    auto fetch = [&](int blk) {
        Block<DK, R> &x = blocks[blk % kBlocks];
        const int t = t_lo + blk * kTokens, n = min(kTokens, t_hi - t);
        for (int i = tid; i < n * (DK / 4); i += kThreads) {
            const int tt = i / (DK / 4), c = i % (DK / 4) * 4;
            copy16(&x.k[tt][c], kb + (t + tt) * k_step + c);
            if constexpr (!kStateOnly) copy16(&x.q[tt][c], qb + (t + tt) * k_step + c);
        }
        for (int i = tid; i < n * (kRows / 4); i += kThreads) {
            const int tt = i / (kRows / 4), c = i % (kRows / 4) * 4;
            copy16(&x.v[tt][c], vb + (t + tt) * v_step + c);
        }
        if (tid < n) x.alpha[tid] = a_next;
    };
    for (int i = 0; i < 2; ++i) {
        if (i < n_blocks) {
            fetch_alpha(i);
            fetch(i);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    if (2 < n_blocks) fetch_alpha(2);

    clear();
    if (g == 0) {
        const float *s0 = initial_state_ptr(p.s0, p.s0_idx, p.n_s0, b, h, Hv, dv, DK, p.err);
        if (s0 != nullptr) add_rows(s0, 0.f);
    } else if constexpr (!kStateOnly) {
        for (int s = 0; s < g; ++s) add_rows(p.seg_state + (seg0 + s) * mat, p.seg_decay[seg0 + s]);
    }
    float kept = 1.f;
    for (int blk = 0; blk < n_blocks; ++blk) {
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();  // this block is there, and the one before is done with
        if (blk + 2 < n_blocks) fetch(blk + 2);
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (blk + 3 < n_blocks) fetch_alpha(blk + 3);
        const Block<DK, R> &x = blocks[blk % kBlocks];
        const int t = t_lo + blk * kTokens, n = min(kTokens, t_hi - t);
        for (int i0 = 0; i0 < n; i0 += 4) {
            float part[4 * R];  // [row][token] of this lane's columns
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int i = i0 + j;
                if (i < n) {
                    const float a = x.alpha[i];
                    const float2 a2 = make_float2(a, a);
                    if constexpr (kStateOnly) kept *= a;
                    float2 v2[R], acc[R];
#pragma unroll
                    for (int r = 0; r < R; r += 2) {
                        const float2 v = *reinterpret_cast<const float2 *>(&x.v[i][row0 + r]);
                        v2[r] = make_float2(v.x, v.x);
                        v2[r + 1] = make_float2(v.y, v.y);
                        acc[r] = acc[r + 1] = make_float2(0.f, 0.f);
                    }
#pragma unroll
                    for (int f = 0; f < F2 / 2; ++f) {
                        const float4 k4 = *reinterpret_cast<const float4 *>(&x.k[i][(f * 8 + l8) * 4]);
                        const float2 k2[2] = {make_float2(k4.x, k4.y), make_float2(k4.z, k4.w)};
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                S[r][2 * f + e] = __ffma2_rn(a2, S[r][2 * f + e], __fmul2_rn(v2[r], k2[e]));
                        if constexpr (!kStateOnly) {
                            const float4 q4 = *reinterpret_cast<const float4 *>(&x.q[i][(f * 8 + l8) * 4]);
                            const float2 q2[2] = {make_float2(q4.x, q4.y), make_float2(q4.z, q4.w)};
#pragma unroll
                            for (int r = 0; r < R; ++r)
#pragma unroll
                                for (int e = 0; e < 2; ++e) acc[r] = __ffma2_rn(S[r][2 * f + e], q2[e], acc[r]);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r) part[r * 4 + j] = acc[r].x + acc[r].y;
                } else {
                    #pragma unroll
                    for (int r = 0; r < R; ++r) part[r * 4 + j] = 0.f;
                }
            }
            if constexpr (!kStateOnly) {
                // reduce-scatter over the rows' eight lanes: lane l8 ends with the sums of
                // the values [row][token] from l8 R / 2 on
#pragma unroll
                for (int o = 4, m = 2 * R; o > 0; o >>= 1, m >>= 1) {
                    const bool up = (l8 & o) != 0;
#pragma unroll
                    for (int e = 0; e < m; ++e) {
                        const float give = up ? part[e] : part[e + m], keep = up ? part[e + m] : part[e];
                        part[e] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                    }
                }
#pragma unroll
                for (int e = 0; e < R / 2; ++e) {
                    const int at = l8 * (R / 2) + e, i = i0 + (at & 3);
                    if (i < n) ob[(long)(t + i) * v_step + row0 + (at >> 2)] = p.scale * part[e];
                }
            }
        }
    }
    if constexpr (kStateOnly) {
        store_rows(p.seg_state + (seg0 + g) * mat);
        if (tid == 0 && tile == 0) p.seg_decay[seg0 + g] = kept;
    } else if (p.s_final != nullptr && g == 0) {
        if (p.G > 1) {  // the row's last state, from the segments' (see the tensor-core path)
            clear();
            for (int s = 0; s < p.G; ++s) add_rows(p.seg_state + (seg0 + s) * mat, p.seg_decay[seg0 + s]);
        }
        store_rows(p.s_final + ((size_t)b * Hv + h) * mat);
    }
}

// Rows a lane: four where a CTA's 64 divide dv (half the key and query loads from
// shared memory, which bound two rows), else two.
int rows_of(int dv) { return dv % 64 == 0 ? 64 : 32; }

// Segments a row: as many as fill three CTAs on every SM, of 64 tokens at least, where
// that makes four or more.  The first pass costs two thirds of the work again, and three
// CTAs on an SM take 2.2 times as long as one: at dk = dv = 128, 32 heads and 4100 tokens
// took 832 us as one segment, 535 as 4, 431 as 7; two rows of 2048: 420 us, 498 as 3.
int segments(int B, int T, int Hv, int dv, bool varlen) {
    const long slots = 3l * sm_count_of_current_device(), units = (long)B * Hv * (dv / rows_of(dv));
    if (units == 0) return 1;
    const long longest = varlen ? (T + B - 1) / B : T;  // packed rows: their mean
    long g = slots / units;
    if (g > longest / 64) g = longest / 64;
    return g < 4 ? 1 : (int)g;
}

template <int DK, int R>
cudaError_t launch_dk(F32Params p, cudaStream_t stream) {
    constexpr int bytes = kBlocks * (int)sizeof(Block<DK, R>);
    const long units = (long)p.B * p.Hv * (p.dv / (16 * R));
    if (units * p.G > 0x7fffffffL) return cudaErrorInvalidValue;
    cudaError_t e = set_smem_once<linear_f32_kernel<DK, R, false>>(bytes);
    if (e != cudaSuccess) return e;
    if (p.G > 1) {
        e = set_smem_once<linear_f32_kernel<DK, R, true>>(bytes);
        if (e != cudaSuccess) return e;
        // the last segment's end state is only needed for the final state
        p.G_run = p.s_final != nullptr ? p.G : p.G - 1;
        linear_f32_kernel<DK, R, true><<<(unsigned)(units * p.G_run), kThreads, bytes, stream>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    p.G_run = p.G;
    linear_f32_kernel<DK, R, false><<<(unsigned)(units * p.G), kThreads, bytes, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t linear_f32_workspace_bytes(int B, int T, int Hv, int dk, int dv, bool varlen) {
    const int G = segments(B, T, Hv, dv, varlen);
    return G == 1 ? 0 : (size_t)B * Hv * G * ((size_t)dv * dk + 1) * sizeof(float);
}

cudaError_t launch_linear_f32(const PrefillParams &pp, cudaStream_t stream) {
    F32Params p{};
    static_cast<PrefillParams &>(p) = pp;
    p.G = segments(p.B, p.T, p.Hv, p.dv, p.cu_seqlens != nullptr);
    if (p.G > 1) {
        p.seg_state = reinterpret_cast<float *>(p.ws);
        p.seg_decay = p.seg_state + (size_t)p.B * p.Hv * p.G * p.dv * p.dk;
    }
    const bool four = rows_of(p.dv) == 64;
    switch (p.dk) {
        case 32: return four ? launch_dk<32, 4>(p, stream) : launch_dk<32, 2>(p, stream);
        case 64: return four ? launch_dk<64, 4>(p, stream) : launch_dk<64, 2>(p, stream);
        default: return four ? launch_dk<128, 4>(p, stream) : launch_dk<128, 2>(p, stream);
    }
}

}  // namespace gdn
