// gdn_linear_tc.cu -- linear attention with a decay for each head, chunked
// form on the 5th-generation tensor cores (tcgen05 MMA, TMEM, TMA), for 16-bit
// inputs and dk, dv in {32, 64, 128}.
//
// Per (row, value head), chunk of n <= 64 tokens, start state S0, log2 decays
// a_t, inclusive sums b_t = a_0 + .. + a_t, suffix sums s_t = a_{t+1} + .. + a_63:
//   P[i][j] = 2^{b_i - b_j} scale q_i.k_j   (j <= i, else 0)
//   O       = P V + diag(scale 2^{b_i}) Q S0^T
//   S_end   = 2^{b_63} S0 + W^T K,   W[t] = 2^{s_t} v_t
// Everything is computed with the value features along the lanes of TMEM:
//   R   = [K;Q] K^T             (lanes 64-127: Q K^T, the raw scores)
//   O1^T = V^T P^T, O2^T = S Q^T, dS = W^T K     (lane = value feature)
// so the state's row, its image as an MMA operand (TMEM), the scaled values W
// (TMEM) and the outputs of one value feature belong to one lane; values and
// outputs are transposed by ldmatrix and stmatrix on their way.
//
// Precision.  The state stays in fp32 registers.  W is given to the MMAs as a
// sum of 16-bit parts: bf16 values split by truncation into three parts hold
// all 24 bits of w v (two parts, 2^-17, where the state is only read by 16-bit
// outputs); fp16 ones into two (22 bits).  P and the state's MMA image are
// rounded to the inputs' type once each, which is the outputs' own rounding
// again.  With fp16, W and the image are scaled per lane, and P per token, by
// powers of two, so neither small nor large states leave fp16's range.
//
// What bounds it: each chunk and head moves 64 KB and takes 1408 tensor cycles
// a SM (256 R, 128 O1, 256 O2, 768 dS) against about 2100 of its share of HBM
// bandwidth, so the loads bound a full grid as long as the tensor pipe never
// waits for the threads.  One persistent CTA a SM, warp-specialised, four
// stages of tiles in flight; every hand-off between the roles is an mbarrier:
//   warps 0-3   state: dS -> fp32 registers -> the next chunk's image
//   warps 4-7   W: values (ldmatrix, transposed), scaled and split, -> TMEM
//   warps 8-11  outputs: O1 + 2^{b} O2, transposed through shared memory (stmatrix), TMA stores
//   warp 12     tiles (TMA) and the chunk's decay sums
//   warp 13     issues every MMA, in the order dS, O2, O1 of a chunk, then R of
//               the next one: the threads' part of each product is done while
//               the others run
//   warps 14-15 P
// Few rows are cut into segments of whole chunks, so that every SM has one: a
// first pass (kStateOnly) forms each segment's end state from its start on,
// and the second takes each segment's start state from those.
//
// Ragged chunks: tokens past the row's end get decay 1 and W = 0, and their K
// and V rows are zeroed in shared memory, so that nothing of the next row (NaN
// and infinities included) enters a product.
//
// Every wait is bounded; on timeout the CTA raises GDN_DEVERR_TIMEOUT, waits
// (bounded) for its copies and MMAs in flight, releases its TMEM and exits.
#include <cstring>

#include "gdn_internal.cuh"
#include "tc_ptx.cuh"

namespace gdn {

// Maps of a [total_T, H, width] 16-bit tensor: tiles of 64 tokens of 64
// features (128-byte swizzle) to load, of 32 features (64-byte swizzle) to store.
bool encode_token_map(CUtensorMap *m, const void *ptr, int H, long total_T, bool bf16, int width);
bool encode_store_map(CUtensorMap *m, void *ptr, int H, long total_T, bool bf16, int width);

namespace {

using namespace tc;

constexpr int C = 64;        // chunk
constexpr int NS = 4;        // stages
constexpr int kThreads = 512;

// Shared memory: per stage two blocks (dk 0-63, 64-127) of [K 64 rows | Q 64
// rows] and two blocks of V; then P, the outputs, the stages' decay sums, the power-of-two
// scales (fp16) and the barriers.
constexpr uint32_t kBlock = 16384;
constexpr uint32_t kStageV = 2 * kBlock;
constexpr uint32_t kStage = kStageV + 16384;
constexpr uint32_t oP = NS * kStage;
constexpr uint32_t oOut = oP + 8192;               // [4 warps][64 tokens][32 features] on their way out
constexpr uint32_t oGate = oOut + 16384;           // per stage: b, scale 2^b, 2^s (64 floats each), 2^b_63
constexpr uint32_t kGate = 1024;
constexpr uint32_t oWInv = oGate + NS * kGate;     // [2][128] 1 / scale of a lane of W
constexpr uint32_t oSInv = oWInv + 1024;           // [2][128] 1 / scale of a lane of the image
constexpr uint32_t oPInv = oSInv + 1024;           // [2][64]  1 / scale of a row of P
constexpr uint32_t oBar = oPInv + 512;
constexpr uint32_t kSmem = oBar + 256 + 1024;      // + alignment slack

// TMEM columns
constexpr uint32_t tR = 0, tO1 = 64, tO2 = 128, tDS = 192, tS = 320, tW = 384;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kBarW = 1;  // named barrier: the W warps

enum Mode {
    kWhole,      // a unit is a whole row: outputs and final state
    kStateOnly,  // a segment's end state from a start of zeros (the first one: from the initial state)
    kOutputs     // a segment's outputs, from the end states before it
};

struct LinearParams : PrefillParams {
    int G;             // segments a row
    int G_run;         // segments of this pass
    float *seg_state;  // [B, Hv, G, dv, dk]
    float *seg_decay;  // [B, Hv, G]
};

template <typename E>
struct Half16;
template <>
struct Half16<__nv_bfloat16> {
    static constexpr bool kBf16 = true;
    __device__ static float2 unpack2(uint32_t u) {
        return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
    }
    __device__ static uint32_t pack2(float a, float b) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
};
template <>
struct Half16<__half> {
    static constexpr bool kBf16 = false;
    __device__ static uint32_t pack2(float a, float b) {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
    __device__ static float2 unpack2(uint32_t u) { return __half22float2(*reinterpret_cast<__half2 *>(&u)); }
};

// A power of two that brings a largest magnitude m into [2^13, 2^14), and its
// inverse (fp16 holds 2^-14 .. 2^15 in full precision).
__device__ __forceinline__ void half_scale(float m, float &s, float &inv) {
    int e = 13 + 127 - (int)(__float_as_uint(m) >> 23);
    e = e > 126 ? 126 : (e < -126 ? -126 : e);
    if (!(m > 0.f)) e = 0;
    s = __uint_as_float((uint32_t)(127 + e) << 23);
    inv = __uint_as_float((uint32_t)(127 - e) << 23);
}

// One unit: a segment of a (row, value head).
struct Unit {
    int b, h, g, len, c0, c1;
    long tok0;
};
__device__ __forceinline__ Unit unit_at(const LinearParams &p, long u) {
    Unit x;
    const unsigned r = (unsigned)((unsigned long)u / (unsigned)p.Hv);
    x.h = (int)(u - (long)r * p.Hv);
    x.b = (int)(r / (unsigned)p.G_run);
    x.g = (int)(r - (unsigned)x.b * (unsigned)p.G_run);
    row_range(p.cu_seqlens, x.b, p.T, x.tok0, x.len);
    const int nc = (x.len + C - 1) / C, per = (nc + p.G - 1) / p.G;
    x.c0 = min(x.g * per, nc);
    x.c1 = min(x.c0 + per, nc);
    return x;
}
__device__ __forceinline__ long n_units(const LinearParams &p) { return (long)p.B * p.Hv * p.G_run; }

// The CTA's chunks, unit after unit.
struct Cursor {
    long u;
    int c;
    Unit x;
    __device__ __forceinline__ void start() {
        u = (long)blockIdx.x - gridDim.x;
        c = 0;
        x.c1 = 0;
    }
    __device__ __forceinline__ bool next(const LinearParams &p) {
        ++c;
        while (c >= x.c1) {
            u += gridDim.x;
            if (u >= n_units(p)) return false;
            x = unit_at(p, u);
            c = x.c0;
        }
        return true;
    }
};

template <typename E, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
linear_kernel(const LinearParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
              const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
    using H = Half16<E>;
    constexpr bool kBf = H::kBf16;
    constexpr bool kOut = MODE != kStateOnly;
    constexpr int NT = kBf && MODE != kOutputs ? 3 : 2;  // 16-bit parts of W
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_align1k(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + oBar), *empty = full + NS;
    uint64_t *r_done = empty + NS, *r_free = r_done + 1, *p_ready = r_done + 2, *w_ready = r_done + 3,
             *ds_done = r_done + 4, *ds_free = r_done + 5, *qs_done = r_done + 6, *s_ready = r_done + 7,
             *o_done = r_done + 8, *o_free = r_done + 9, *drain = r_done + 10;
    uint32_t *slot = reinterpret_cast<uint32_t *>(r_done + 11);
    // (through a shuffle: known to be the same in every lane)
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int dk = p.dk, dv = p.dv, Hv = p.Hv, Hk = p.Hk;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 2);                  // the copies' thread, the decay sums
            mbar_init(&empty[s], kOut ? 1 + 4 + 4 : 1 + 4);  // MMAs, state warps, output warps
        }
        mbar_init(r_done, 1);
        mbar_init(r_free, 2);
        mbar_init(p_ready, 2);
        mbar_init(w_ready, 4);
        mbar_init(ds_done, 1);
        mbar_init(ds_free, 4);
        mbar_init(qs_done, 1);
        mbar_init(s_ready, 4);
        mbar_init(o_done, 1);
        mbar_init(o_free, 4);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(slot, kTmemCols);
        tmem_relinquish();
    }
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = __shfl_sync(0xffffffffu, *slot, 0);
    bool ok = true;
    // A wait of a whole warp: the outcome is the same in every lane, so that
    // the warp-wide TMEM accesses behind it stay converged.
    auto wait = [&](uint64_t *bar, int it) {
        const bool done = mbar_wait(bar, (uint32_t)it & 1u, p.wait_ns);
        return __all_sync(0xffffffffu, done) != 0;
    };
    auto wait_full = [&](int it) { return wait(&full[it % NS], it / NS); };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    if (warp < 4) {
        // ============================ state ==============================
        regs_inc<200>();
        const int i = warp * 32 + lane;  // value feature
        const uint32_t lane_base = tm + ((uint32_t)(warp * 32) << 16);
        const float *winv = reinterpret_cast<const float *>(sm + oWInv);
        float *sinv = reinterpret_cast<float *>(sm + oSInv);
        float2 S[64];  // columns 2 j, 2 j + 1
        int it = 0;
        const size_t mat = (size_t)dv * dk;
        auto clear = [&]() {
#pragma unroll
            for (int j = 0; j < 64; ++j) S[j] = make_float2(0.f, 0.f);
        };
        auto add_row = [&](const float *src, float keep) {  // S <- keep S + row i
            const float2 k2 = make_float2(keep, keep);
#pragma unroll
            for (int q = 0; q < 32; ++q) {
                if (q * 4 < dk) {
                    const float4 f = *reinterpret_cast<const float4 *>(src + (size_t)i * dk + q * 4);
                    S[2 * q] = __ffma2_rn(k2, S[2 * q], make_float2(f.x, f.y));
                    S[2 * q + 1] = __ffma2_rn(k2, S[2 * q + 1], make_float2(f.z, f.w));
                }
            }
        };
        // S <- the state after the row's segments s < n (nothing yet if 0)
        auto fold = [&](size_t seg0, int n) {
#pragma unroll 1
            for (int s = 0; s < n; ++s) add_row(p.seg_state + (seg0 + s) * mat, p.seg_decay[seg0 + s]);
        };
        for (long u = blockIdx.x; ok && u < n_units(p); u += gridDim.x) {
            const Unit x = unit_at(p, u);
            const size_t seg0 = ((size_t)x.b * Hv + x.h) * p.G;
            clear();
            if (x.g == 0) {
                const float *s0 = initial_state_ptr(p.s0, p.s0_idx, p.n_s0, x.b, x.h, Hv, dv, dk, p.err);
                if (s0 != nullptr && i < dv) add_row(s0, 0.f);
            } else if (MODE == kOutputs && i < dv) {
                fold(seg0, x.g);
            }
            float kept = 1.f;  // the segment's decay
#pragma unroll 1
            for (int c = x.c0; c < x.c1; ++c, ++it) {
                if constexpr (kOut) {
                    // this chunk's start state as an MMA operand
                    float sc = 1.f;
                    if constexpr (!kBf) {
                        float m = 0.f, inv;
#pragma unroll
                        for (int j = 0; j < 64; ++j) m = fmaxf(m, fmaxf(fabsf(S[j].x), fabsf(S[j].y)));
                        half_scale(m, sc, inv);
                        sinv[(it & 1) * 128 + i] = inv;
                    }
                    if (it > 0 && !(ok = wait(qs_done, it - 1))) break;
                    fence_after_sync();
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        if (g * 32 < dk) {
                            uint32_t v[16];
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                v[j] = kBf ? H::pack2(S[16 * g + j].x, S[16 * g + j].y)
                                           : H::pack2(sc * S[16 * g + j].x, sc * S[16 * g + j].y);
                            tmem_st16(lane_base + tS + 16 * g, v);
                        }
                    }
                    tmem_wait_st();
                    fence_before_sync();
                    arrive(s_ready);
                }
                // S <- 2^b_63 S + dS
                if (!(ok = wait_full(it)) || !(ok = wait(ds_done, it))) break;
                fence_after_sync();
                const float gam = reinterpret_cast<const float *>(sm + oGate + (it % NS) * kGate)[192];
                const float wi = kBf ? 1.f : winv[(it & 1) * 128 + i];
                const float2 gam2 = make_float2(gam, gam), wi2 = make_float2(wi, wi);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (g * 32 < dk) {
                        float v[32];
                        tmem_ld32(lane_base + tDS + 32 * g, v);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float2 d = make_float2(v[2 * j], v[2 * j + 1]);
                            if constexpr (!kBf) d = __fmul2_rn(wi2, d);
                            S[16 * g + j] = __ffma2_rn(gam2, S[16 * g + j], d);
                        }
                    }
                }
                kept *= gam;
                fence_before_sync();
                arrive(ds_free);
                arrive(&empty[it % NS]);
            }
            if (!ok) break;
            float *dst = nullptr;
            if (MODE == kStateOnly) {
                dst = p.seg_state + (seg0 + x.g) * mat;
                if (i == 0) p.seg_decay[seg0 + x.g] = kept;
            } else if (p.s_final != nullptr && x.g == 0) {
                // with segments, the row's last state from theirs (this thread
                // has read its row of the initial state: final may replace it)
                dst = p.s_final + ((size_t)x.b * Hv + x.h) * mat;
                if (MODE == kOutputs && i < dv) {
                    clear();
                    fold(seg0, p.G);
                }
            }
            if (dst != nullptr && i < dv) {
#pragma unroll
                for (int q = 0; q < 32; ++q)
                    if (q * 4 < dk)
                        *reinterpret_cast<float4 *>(dst + (size_t)i * dk + q * 4) =
                            make_float4(S[2 * q].x, S[2 * q].y, S[2 * q + 1].x, S[2 * q + 1].y);
            }
        }
    } else if (warp < 8) {
        // ============================== W ================================
        const int wq = warp - 4, tid = threadIdx.x - 128;
        const uint32_t lane_base = tm + ((uint32_t)(wq * 32) << 16);
        float *winv = reinterpret_cast<float *>(sm + oWInv);
        // ldmatrix: this lane's row of the four 8 x 8 matrices (tokens 0-7 and
        // 8-15 of 16, features 0-7 and 8-15 of 16)
        const int row = (lane & 7) + ((lane >> 4) << 3), cg = (wq & 1) * 4 + ((lane >> 3) & 1);
        const uint32_t v_off = kStageV + (wq >> 1) * 8192 + row * 128;
        Cursor k;
        k.start();
#pragma unroll 1
        for (int it = 0; k.next(p); ++it) {
            const int n = min(C, k.x.len - k.c * C);
            if (!(ok = wait_full(it))) break;
            uint8_t *st = sm + (it % NS) * kStage;
            const float *w = reinterpret_cast<const float *>(sm + oGate + (it % NS) * kGate) + 128 + 2 * (lane & 3);
            if (n < C) {
                // K and V rows past the row's end: zeros, whatever was loaded
#pragma unroll 1
                for (int e = tid; e < (C - n) * 8; e += 128) {
                    const int r = n + (e >> 3), off = r * 128 + (e & 7) * 16;
                    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4 *>(st + off) = z;
                    *reinterpret_cast<uint4 *>(st + kBlock + off) = z;
                    *reinterpret_cast<uint4 *>(st + kStageV + off) = z;
                    *reinterpret_cast<uint4 *>(st + kStageV + 8192 + off) = z;
                }
                fence_proxy_async();
                named_bar(kBarW, 128);
            }
            // 16 features at a time: lanes g and g + 8 of them, tokens 2 t, 2 t + 1
            // of each eight, in the layout of the TMEM store
#pragma unroll 1
            for (int hh = 0; hh < 2; ++hh) {
                uint32_t part[NT][16];
                float2 x[16];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t v[4];
                    ldsm_x4_trans(v, st + v_off + j * 2048 + (((cg + 2 * hh) ^ (lane & 7)) << 4));
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 w2 = *reinterpret_cast<const float2 *>(w + 16 * j + 8 * (e >> 1));
                        x[4 * j + e] = __fmul2_rn(w2, H::unpack2(v[e]));
                    }
                }
                if constexpr (kBf) {
                    // the upper 16 bits are a bf16 by truncation; what is left is exact
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float2 r = x[e];
#pragma unroll
                        for (int m = 0; m < NT - 1; ++m) {
                            const uint32_t a = __float_as_uint(r.x), b = __float_as_uint(r.y);
                            part[m][e] = __byte_perm(a, b, 0x7632);
                            r = __fadd2_rn(r, make_float2(__uint_as_float((a & 0xffff0000u) ^ 0x80000000u),
                                                          __uint_as_float((b & 0xffff0000u) ^ 0x80000000u)));
                        }
                        part[NT - 1][e] = H::pack2(r.x, r.y);
                    }
                } else {
                    // the largest magnitude of each of the two features, over its
                    // four lanes, gives its scale
                    float m0 = 0.f, m1 = 0.f, s0, s1, i0, i1;
#pragma unroll
                    for (int e = 0; e < 16; e += 2) {
                        m0 = fmaxf(m0, fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
                        m1 = fmaxf(m1, fmaxf(fabsf(x[e + 1].x), fabsf(x[e + 1].y)));
                    }
#pragma unroll
                    for (int o = 1; o < 4; o <<= 1) {
                        m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
                        m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
                    }
                    half_scale(m0, s0, i0);
                    half_scale(m1, s1, i1);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float s = (e & 1) ? s1 : s0;
                        const float2 y = __fmul2_rn(make_float2(s, s), x[e]);
                        part[0][e] = H::pack2(y.x, y.y);
                        const float2 h = H::unpack2(part[0][e]);
                        part[1][e] = H::pack2(y.x - h.x, y.y - h.y);
                    }
                    if (hh == 0 && it > 0 && !(ok = wait(ds_done, it - 1))) break;
                    if ((lane & 3) == 0) {
                        winv[(it & 1) * 128 + wq * 32 + 16 * hh + (lane >> 2)] = i0;
                        winv[(it & 1) * 128 + wq * 32 + 16 * hh + (lane >> 2) + 8] = i1;
                    }
                }
                if (kBf && hh == 0 && it > 0 && !(ok = wait(ds_done, it - 1))) break;
                fence_after_sync();
#pragma unroll
                for (int m = 0; m < NT; ++m) tmem_st_16x32(lane_base + ((uint32_t)(16 * hh) << 16) + tW + 32 * m, part[m]);
            }
            if (!ok) break;
            tmem_wait_st();
            fence_before_sync();
            arrive(w_ready);
        }
    } else if (warp < 12) {
        // ============================ outputs ============================
        regs_dec<96>();
        if constexpr (kOut) {
            const int wq = warp - 8;
            const uint32_t lane_base = tm + ((uint32_t)(wq * 32) << 16);
            const float *sinv = reinterpret_cast<const float *>(sm + oSInv) + wq * 32 + (lane >> 2);
            const float *pinv = reinterpret_cast<const float *>(sm + oPInv) + 2 * (lane & 3);
            uint8_t *buf = sm + oOut + wq * 4096;  // [64 tokens][32 features], 64-byte swizzle
            // stmatrix: this lane's row (token) of the four 8 x 8 matrices (features
            // 0-7 and 8-15 of 16, tokens 0-7 and 8-15 of 16)
            const int row = (lane & 7) + ((lane >> 4) << 3), cg = (lane >> 3) & 1;
            const bool mine = wq * 32 < dv;
            Cursor k;
            k.start();
#pragma unroll 1
            for (int it = 0; k.next(p); ++it) {
                const int n = min(C, k.x.len - k.c * C);
                if (!(ok = wait_full(it)) || !(ok = wait(o_done, it))) break;
                fence_after_sync();
                const float *eb = reinterpret_cast<const float *>(sm + oGate + (it % NS) * kGate) + 64 + 2 * (lane & 3);
                if (lane == 0) bulk_wait_read_all();  // the last chunk's tile has left
                __syncwarp();
#pragma unroll 1
                for (int part = 0; part < 4; ++part) {
                    const int hh = part & 1, th = part >> 1;  // 16 features, 32 tokens
                    uint32_t o1[16], o2[16];
                    tmem_ld_16x32(lane_base + ((uint32_t)(16 * hh) << 16) + tO1 + 32 * th, o1);
                    tmem_ld_16x32(lane_base + ((uint32_t)(16 * hh) << 16) + tO2 + 32 * th, o2);
                    tmem_wait_ld();
                    uint32_t v[8];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float2 e2 = *reinterpret_cast<const float2 *>(eb + 32 * th + 8 * r);
                        float2 p2 = make_float2(1.f, 1.f);
                        if constexpr (!kBf) p2 = *reinterpret_cast<const float2 *>(pinv + (it & 1) * 64 + 32 * th + 8 * r);
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            float2 a = make_float2(__uint_as_float(o1[4 * r + 2 * m]), __uint_as_float(o1[4 * r + 2 * m + 1]));
                            const float2 b =
                                make_float2(__uint_as_float(o2[4 * r + 2 * m]), __uint_as_float(o2[4 * r + 2 * m + 1]));
                            float2 e = e2;
                            if constexpr (!kBf) {
                                const float si = sinv[(it & 1) * 128 + 16 * hh + 8 * m];
                                e = __fmul2_rn(e, make_float2(si, si));
                                a = __fmul2_rn(a, p2);
                            }
                            const float2 o = __ffma2_rn(e, b, a);
                            v[2 * r + m] = H::pack2(o.x, o.y);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < 2; ++r) {
                        const int t = 32 * th + 16 * r + row;
                        const uint32_t f[4] = {v[4 * r], v[4 * r + 1], v[4 * r + 2], v[4 * r + 3]};
                        stsm_x4_trans(buf + t * 64 + (((2 * hh + cg) ^ ((t >> 1) & 3)) << 4), f);
                    }
                }
                fence_before_sync();
                arrive(o_free);
                arrive(&empty[it % NS]);
                const long t0 = k.x.tok0 + (long)k.c * C;
                if (mine && n == C) {
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&mo, wq * 32, k.x.h, (int)t0, buf);
                        bulk_commit();
                    }
                } else if (mine) {  // the next row's tokens stay untouched
                    __syncwarp();
#pragma unroll 1
                    for (int e = lane; e < n * 4; e += 32) {
                        const int t = e >> 2, q = e & 3;
                        *reinterpret_cast<uint4 *>(reinterpret_cast<E *>(p.out) + ((t0 + t) * Hv + k.x.h) * dv + wq * 32 + 8 * q) =
                            *reinterpret_cast<const uint4 *>(buf + t * 64 + ((q ^ ((t >> 1) & 3)) << 4));
                    }
                    __syncwarp();
                }
            }
            if (lane == 0) bulk_wait_all();
        }
    } else {
        regs_dec<88>();
        if (warp == 12) {
            // ====================== tiles, decay sums ====================
            int issued = 0;
            Cursor k;
            k.start();
            const bool per_head = (p.conv & GDN_ALPHA_PER_HEAD) != 0;
            float raw[2] = {0.f, 0.f};
            auto fetch = [&]() {  // the chunk's decays of tokens 2 lane, 2 lane + 1 as they are stored
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int t = k.c * C + 2 * lane + e;
                    if (t < k.x.len)
                        raw[e] = ld_gate_early(p.alpha, per_head ? (long)k.x.h : (k.x.tok0 + t) * Hv + k.x.h, p.dt_gate);
                }
            };
            bool more = k.next(p);
            if (more) fetch();
            for (int it = 0; more; ++it) {
                const int s = it % NS;
                uint8_t *st = sm + s * kStage;
                if (it >= NS && !(ok = wait(&empty[s], it / NS - 1))) break;
                if (lane == 0) {
                    const int hk = k.x.h / (Hv / Hk), t0 = (int)(k.x.tok0 + (long)k.c * C);
                    const int kb = dk > 64 ? 2 : 1, vb = dv > 64 ? 2 : 1;
                    mbar_arrive_expect_tx(&full[s], 8192u * (kb * (kOut ? 2 : 1) + vb));
                    for (int j = 0; j < kb; ++j) {
                        tma_load_3d(st + j * kBlock, &mk, 64 * j, hk, t0, &full[s]);
                        if constexpr (kOut) tma_load_3d(st + j * kBlock + 8192, &mq, 64 * j, hk, t0, &full[s]);
                    }
                    for (int j = 0; j < vb; ++j) tma_load_3d(st + kStageV + j * 8192, &mv, 64 * j, k.x.h, t0, &full[s]);
                }
                ++issued;
                float a[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    a[e] = (p.conv & GDN_ALPHA_LOG) ? raw[e] * kLog2e : log2f(raw[e]);
                    if (k.c * C + 2 * lane + e >= k.x.len) a[e] = 0.f;
                }
                more = k.next(p);
                if (more) fetch();
                // inclusive sums over the lanes from both ends; the exclusive ones
                // are the neighbours' (a difference would lose what a strong decay
                // has in front of it, and be no number after a decay of 0)
                auto scan = [&](float v, bool up) {
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const float y = up ? __shfl_up_sync(0xffffffffu, v, o) : __shfl_down_sync(0xffffffffu, v, o);
                        if (up ? lane >= o : lane + o < 32) v += y;
                    }
                    return v;
                };
                float *gate = reinterpret_cast<float *>(sm + oGate + s * kGate);
                const float inc = scan(a[0] + a[1], true);
                float ex = __shfl_up_sync(0xffffffffu, inc, 1);
                if (lane == 0) ex = 0.f;
                float suf = __shfl_down_sync(0xffffffffu, scan(a[0] + a[1], false), 1);
                if (lane == 31) suf = 0.f;
                float2 bc = make_float2(ex + a[0], inc);
                gate[64 + 2 * lane] = p.scale * exp2f(bc.x);
                gate[64 + 2 * lane + 1] = p.scale * exp2f(bc.y);
                gate[128 + 2 * lane] = exp2f(suf + a[1]);
                gate[128 + 2 * lane + 1] = exp2f(suf);
                if (lane == 31) gate[192] = exp2f(inc);
                // For P's differences a decay below 2^-40 (0 among them) counts as
                // 2^-40, far below the scores' own rounding: the sums stay finite,
                // and small enough for their differences to be exact to 2^-12.
                const bool strong = a[0] < -40.f || a[1] < -40.f;
                if (__any_sync(0xffffffffu, strong)) {
                    const float c0 = a[0] < -40.f ? -40.f : a[0], c1 = a[1] < -40.f ? -40.f : a[1];
                    const float ic = scan(c0 + c1, true);
                    float ec = __shfl_up_sync(0xffffffffu, ic, 1);
                    if (lane == 0) ec = 0.f;
                    bc = make_float2(ec + c0, ic);
                }
                *reinterpret_cast<float2 *>(gate + 2 * lane) = bc;
                arrive(&full[s]);
            }
            if (!ok)  // the copies in flight must land before the CTA ends
                for (int j = issued > NS ? issued - NS : 0; j < issued; ++j)
                    mbar_wait(&full[j % NS], (uint32_t)(j / NS) & 1u, kDefaultWaitNs);
        } else if (warp == 13) {
            // =========================== MMAs ============================
            const uint32_t id_r = idesc_f16(128, 64, false, false, kBf);
            const uint32_t id_o1 = idesc_f16(128, 64, true, false, kBf);
            const uint32_t id_o2 = idesc_f16(128, 64, false, false, kBf);
            const uint32_t id_ds = idesc_f16(128, dk, false, true, kBf);
            const int ks = dk / 16;  // K = 16 steps over dk
            const uint32_t s0 = smem_u32(sm);
            auto raw_scores = [&](int it) {
                if (!wait_full(it) || (it > 0 && !wait(r_free, it - 1))) return false;
                fence_after_sync();
                const uint64_t kq = desc_sw128(s0 + (it % NS) * kStage, 16, 1024);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    if (k >= ks) break;
                    const uint64_t d = desc_add(kq, (k >> 2) * kBlock + (k & 3) * 32);
                    mma_f16_elect(tm + tR, d, d, id_r, k > 0);
                }
                mma_commit_elect(r_done);
                return true;
            };
            Cursor k;
            k.start();
            bool more = k.next(p);
            if constexpr (kOut) ok = !more || raw_scores(0);
#pragma unroll 1
            for (int it = 0; ok && more; ++it) {
                const uint32_t st = s0 + (it % NS) * kStage;
                // dS = W^T K, every part of W
                if (!(ok = wait_full(it)) || !(ok = wait(w_ready, it)) || (it > 0 && !(ok = wait(ds_free, it - 1)))) break;
                fence_after_sync();
                const uint64_t kn = desc_sw128(st, kBlock, 1024);
#pragma unroll
                for (int m = 0; m < NT; ++m)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_f16_ta_elect(tm + tDS, tm + tW + 32 * m + 8 * j, desc_add(kn, j * 2048), id_ds, m + j > 0);
                mma_commit_elect(ds_done);
                if constexpr (kOut) {
                    // O2^T = S Q^T
                    if (!(ok = wait(s_ready, it)) || (it > 0 && !(ok = wait(o_free, it - 1)))) break;
                    fence_after_sync();
                    const uint64_t qd = desc_sw128(st + 8192, 16, 1024);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        if (j >= ks) break;
                        mma_f16_ta_elect(tm + tO2, tm + tS + 8 * j, desc_add(qd, (j >> 2) * kBlock + (j & 3) * 32), id_o2,
                                         j > 0);
                    }
                    mma_commit_elect(qs_done);
                    // O1^T = V^T P^T
                    if (!(ok = wait(p_ready, it))) break;
                    fence_after_sync();
                    const uint64_t vd = desc_sw128(st + kStageV, 8192, 1024), pd = desc_sw128(s0 + oP, 16, 1024);
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        mma_f16_elect(tm + tO1, desc_add(vd, j * 2048), desc_add(pd, j * 32), id_o1, j > 0);
                    mma_commit_elect(o_done);
                }
                mma_commit_elect(&empty[it % NS]);
                more = k.next(p);
                if constexpr (kOut)
                    if (more && !(ok = raw_scores(it + 1))) break;
            }
            mma_commit_elect(drain);  // nothing may be in flight when TMEM is given back
            mbar_wait(drain, 0, kDefaultWaitNs);
        } else {
            // ============================= P =============================
            if constexpr (kOut) {
                const int i = (warp - 14) * 32 + lane;  // token of the chunk
                const uint32_t lane_base = tm + ((uint32_t)(64 + (warp - 14) * 32) << 16);
                float *pinv = reinterpret_cast<float *>(sm + oPInv);
                Cursor k;
                k.start();
                for (int it = 0; k.next(p); ++it) {
                    if (!(ok = wait_full(it)) || !(ok = wait(r_done, it))) break;
                    fence_after_sync();
                    const float *b = reinterpret_cast<const float *>(sm + oGate + (it % NS) * kGate);
                    const float bi = b[i];
                    // 16 columns of the row: zero above the diagonal
                    auto columns = [&](int cb, float (&x)[16]) {
                        tmem_ld16(lane_base + tR + 16 * cb, x);
#pragma unroll
                        for (int j = 0; j < 16; j += 4) {
                            const float4 b4 = *reinterpret_cast<const float4 *>(b + 16 * cb + j);
                            const float bs[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[j + e] = 16 * cb + j + e <= i ? x[j + e] * p.scale * ex2_approx(bi - bs[e]) : 0.f;
                        }
                    };
                    const int blocks = 2 * (warp - 14) + 2;  // the warp's rows end in column 16 blocks - 1
                    float sc = 1.f;
                    if constexpr (!kBf) {
                        float m = 0.f, inv;
#pragma unroll 1
                        for (int cb = 0; cb < blocks; ++cb) {
                            float x[16];
                            columns(cb, x);
#pragma unroll
                            for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(x[j]));
                        }
                        half_scale(m, sc, inv);
                        pinv[(it & 1) * 64 + i] = inv;
                    }
#pragma unroll 1
                    for (int cb = 0; cb < 4; ++cb) {
                        uint32_t v[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
                        if (cb < blocks) {
                            float x[16];
                            columns(cb, x);
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                v[j] = kBf ? H::pack2(x[2 * j], x[2 * j + 1]) : H::pack2(sc * x[2 * j], sc * x[2 * j + 1]);
                        }
                        *reinterpret_cast<uint4 *>(sm + oP + sw128_chunk(i, 2 * cb)) = make_uint4(v[0], v[1], v[2], v[3]);
                        *reinterpret_cast<uint4 *>(sm + oP + sw128_chunk(i, 2 * cb + 1)) = make_uint4(v[4], v[5], v[6], v[7]);
                    }
                    fence_before_sync();
                    arrive(r_free);
                    fence_proxy_async();
                    arrive(p_ready);
                }
            }
        }
    }
    if (!ok && lane == 0) atomicOr(p.err, (uint32_t)GDN_DEVERR_TIMEOUT);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 0) tmem_dealloc(tm, kTmemCols);
}

// Segments a row: 1 as soon as the rows and heads alone give every SM a unit;
// else as many as fit one wave, with two chunks each at least.
int segments(int B, int T, int Hv, bool varlen) {
    const long sms = sm_count_of_current_device(), units = (long)B * Hv;
    if (units == 0 || units * 2 > sms) return 1;
    const long longest = varlen ? (T + B - 1) / B : T;  // packed rows: their mean
    const long chunks = (longest + C - 1) / C;
    long g = sms / units;
    if (g > chunks / 2) g = chunks / 2;
    return g < 2 ? 1 : (int)g;
}

template <typename E, int MODE>
cudaError_t launch_mode(LinearParams p, int g_run, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                        const CUtensorMap &mo, cudaStream_t stream) {
    p.G_run = g_run;
    const long units = (long)p.B * p.Hv * g_run, sms = sm_count_of_current_device();
    if (units == 0) return cudaSuccess;
    cudaError_t e = set_smem_once<linear_kernel<E, MODE>>((int)kSmem);
    if (e != cudaSuccess) return e;
    linear_kernel<E, MODE><<<(unsigned)(units < sms ? units : sms), kThreads, kSmem, stream>>>(p, mq, mk, mv, mo);
    return cudaGetLastError();
}

template <typename E>
cudaError_t launch_e(const LinearParams &p, long total_T, cudaStream_t stream) {
    constexpr bool bf = Half16<E>::kBf16;
    CUtensorMap mq, mk, mv, mo;
    memset(&mq, 0, sizeof(mq));
    memset(&mk, 0, sizeof(mk));
    memset(&mv, 0, sizeof(mv));
    memset(&mo, 0, sizeof(mo));
    if (total_T > 0 && (!encode_token_map(&mq, p.q, p.Hk, total_T, bf, p.dk) ||
                        !encode_token_map(&mk, p.k, p.Hk, total_T, bf, p.dk) ||
                        !encode_token_map(&mv, p.v, p.Hv, total_T, bf, p.dv) ||
                        !encode_store_map(&mo, p.out, p.Hv, total_T, bf, p.dv)))
        return cudaErrorInvalidValue;
    if (p.G == 1) return launch_mode<E, kWhole>(p, 1, mq, mk, mv, mo, stream);
    // the last segment's end state is only needed for the final state
    cudaError_t e = launch_mode<E, kStateOnly>(p, p.s_final != nullptr ? p.G : p.G - 1, mq, mk, mv, mo, stream);
    if (e != cudaSuccess) return e;
    return launch_mode<E, kOutputs>(p, p.G, mq, mk, mv, mo, stream);
}

size_t state_bytes(int B, int Hv, int G, int dk, int dv) { return (size_t)B * Hv * G * dv * dk * sizeof(float); }

}  // namespace

bool linear_tc_supported(int dk, int dv, int dt_qkv) {
    auto width_ok = [](int d) { return d == 32 || d == 64 || d == 128; };
    return width_ok(dk) && width_ok(dv) && (dt_qkv == GDN_BF16 || dt_qkv == GDN_F16);
}

size_t linear_tc_workspace_bytes(int B, int T, int Hv, int dk, int dv, bool varlen) {
    const int G = segments(B, T, Hv, varlen);
    return G == 1 ? 0 : state_bytes(B, Hv, G, dk, dv) + (size_t)B * Hv * G * sizeof(float);
}

cudaError_t launch_linear_tc(const PrefillParams &pp, cudaStream_t stream) {
    LinearParams p{};
    static_cast<PrefillParams &>(p) = pp;
    const bool varlen = p.cu_seqlens != nullptr;
    const long total_T = varlen ? (long)p.T : (long)p.B * p.T;
    p.G = segments(p.B, p.T, p.Hv, varlen);
    if (p.G > 1) {
        p.seg_state = reinterpret_cast<float *>(p.ws);
        p.seg_decay = reinterpret_cast<float *>(static_cast<uint8_t *>(p.ws) + state_bytes(p.B, p.Hv, p.G, p.dk, p.dv));
    }
    return p.dt_qkv == GDN_BF16 ? launch_e<__nv_bfloat16>(p, total_T, stream) : launch_e<__half>(p, total_T, stream);
}

}  // namespace gdn
