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
// (TMEM) and the outputs of one value feature belong to one lane, and nothing
// is transposed through shared memory but P.
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
//   warps 4-7   W: scaled and split values, registers -> TMEM
//   warps 8-11  outputs: O1 + 2^{b} O2 -> global memory
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

bool encode_token_map(CUtensorMap *m, const void *ptr, int H, long total_T, bool bf16, int width);

namespace {

using namespace tc;

constexpr int C = 64;        // chunk
constexpr int NS = 4;        // stages
constexpr int kThreads = 512;

// Shared memory: per stage two blocks (dk 0-63, 64-127) of [K 64 rows | Q 64
// rows] and two blocks of V; then P, the stages' decay sums, the power-of-two
// scales (fp16) and the barriers.
constexpr uint32_t kBlock = 16384;
constexpr uint32_t kStageV = 2 * kBlock;
constexpr uint32_t kStage = kStageV + 16384;
constexpr uint32_t oP = NS * kStage;
constexpr uint32_t oGate = oP + 8192;              // per stage: b, scale 2^b, 2^s (64 floats each), 2^b_63
constexpr uint32_t kGate = 1024;
constexpr uint32_t oWInv = oGate + NS * kGate;     // [2][128] 1 / scale of a lane of W
constexpr uint32_t oSInv = oWInv + 1024;           // [2][128] 1 / scale of a lane of the image
constexpr uint32_t oPInv = oSInv + 1024;           // [2][64]  1 / scale of a row of P
constexpr uint32_t oBar = oPInv + 512;
constexpr uint32_t kSmem = oBar + 256 + 1024;      // + alignment slack

// TMEM columns
constexpr uint32_t tR = 0, tO1 = 64, tO2 = 128, tDS = 192, tS = 320, tW = 384;
constexpr uint32_t kTmemCols = 512;

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
    __device__ static float up(uint16_t u) { return __uint_as_float((uint32_t)u << 16); }
    __device__ static uint32_t pack2(float a, float b) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
};
template <>
struct Half16<__half> {
    static constexpr bool kBf16 = false;
    __device__ static float up(uint16_t u) { return __half2float(__ushort_as_half(u)); }
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
              const __grid_constant__ CUtensorMap mv) {
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
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    const uint32_t tm = *slot;
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
        float S[128];
        int it = 0;
        const size_t mat = (size_t)dv * dk;
        auto load_row = [&](const float *src, float keep) {  // S <- keep S + row i
#pragma unroll
            for (int q = 0; q < 32; ++q) {
                if (q * 4 < dk) {
                    const float4 f = *reinterpret_cast<const float4 *>(src + (size_t)i * dk + q * 4);
                    S[4 * q + 0] = fmaf(keep, S[4 * q + 0], f.x);
                    S[4 * q + 1] = fmaf(keep, S[4 * q + 1], f.y);
                    S[4 * q + 2] = fmaf(keep, S[4 * q + 2], f.z);
                    S[4 * q + 3] = fmaf(keep, S[4 * q + 3], f.w);
                }
            }
        };
        auto store_row = [&](float *dst) {
#pragma unroll
            for (int q = 0; q < 32; ++q)
                if (q * 4 < dk)
                    *reinterpret_cast<float4 *>(dst + (size_t)i * dk + q * 4) =
                        make_float4(S[4 * q], S[4 * q + 1], S[4 * q + 2], S[4 * q + 3]);
        };
        for (long u = blockIdx.x; ok && u < n_units(p); u += gridDim.x) {
            const Unit x = unit_at(p, u);
            const size_t seg0 = ((size_t)x.b * Hv + x.h) * p.G;
#pragma unroll
            for (int j = 0; j < 128; ++j) S[j] = 0.f;
            if (x.g == 0) {
                const float *s0 = initial_state_ptr(p.s0, p.s0_idx, p.n_s0, x.b, x.h, Hv, dv, dk, p.err);
                if (s0 != nullptr && i < dv) load_row(s0, 0.f);
            } else if (MODE == kOutputs && i < dv) {
                for (int s = 0; s < x.g; ++s)
                    load_row(p.seg_state + (seg0 + s) * mat, p.seg_decay[seg0 + s]);
            }
            float kept = 1.f;  // the segment's decay
            for (int c = x.c0; c < x.c1; ++c, ++it) {
                if constexpr (kOut) {
                    // this chunk's start state as an MMA operand
                    float sc = 1.f;
                    if constexpr (!kBf) {
                        float m = 0.f, inv;
#pragma unroll
                        for (int j = 0; j < 128; ++j) m = fmaxf(m, fabsf(S[j]));
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
                                v[j] = kBf ? H::pack2(S[32 * g + 2 * j], S[32 * g + 2 * j + 1])
                                           : H::pack2(sc * S[32 * g + 2 * j], sc * S[32 * g + 2 * j + 1]);
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
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    if (g * 32 < dk) {
                        float v[32];
                        tmem_ld32(lane_base + tDS + 32 * g, v);
#pragma unroll
                        for (int j = 0; j < 32; ++j) S[32 * g + j] = fmaf(gam, S[32 * g + j], kBf ? v[j] : wi * v[j]);
                    }
                }
                kept *= gam;
                fence_before_sync();
                arrive(ds_free);
                arrive(&empty[it % NS]);
            }
            if (!ok) break;
            if constexpr (MODE == kWhole) {
                if (p.s_final != nullptr && i < dv) store_row(p.s_final + ((size_t)x.b * Hv + x.h) * mat);
            } else if constexpr (MODE == kStateOnly) {
                if (i < dv) store_row(p.seg_state + (seg0 + x.g) * mat);
                if (i == 0) p.seg_decay[seg0 + x.g] = kept;
            } else if (x.g == 0 && p.s_final != nullptr && i < dv) {
                // the row's last state, from the segments' (this thread has
                // read its row of the initial state: final may be in its place)
#pragma unroll
                for (int j = 0; j < 128; ++j) S[j] = 0.f;
                for (int s = 0; s < p.G; ++s) load_row(p.seg_state + (seg0 + s) * mat, p.seg_decay[seg0 + s]);
                store_row(p.s_final + ((size_t)x.b * Hv + x.h) * mat);
            }
        }
    } else if (warp < 8) {
        // ============================== W ================================
        const int i = (warp - 4) * 32 + lane;  // value feature
        const uint32_t lane_base = tm + ((uint32_t)((warp - 4) * 32) << 16);
        float *winv = reinterpret_cast<float *>(sm + oWInv);
        Cursor k;
        k.start();
        for (int it = 0; k.next(p); ++it) {
            const int n = min(C, k.x.len - k.c * C);
            if (!(ok = wait_full(it))) break;
            uint8_t *st = sm + (it % NS) * kStage;
            const uint8_t *vcol = st + kStageV + (i >> 6) * 8192 + (i & 7) * 2;
            const int q = (i & 63) >> 3;
            const float *w = reinterpret_cast<const float *>(sm + oGate + (it % NS) * kGate) + 128;
            // value t of this lane, scaled (0 past the row's end)
            auto wv = [&](int t, float wt) {
                const uint16_t v = *reinterpret_cast<const uint16_t *>(vcol + t * 128 + ((q ^ (t & 7)) << 4));
                return t < n ? wt * H::up(v) : 0.f;
            };
            if (n < C) {
                // K and V rows past the row's end: zeros, whatever was loaded
                const int tid = threadIdx.x - 128;
                for (int e = tid; e < (C - n) * 8; e += 128) {
                    const int r = n + (e >> 3), off = r * 128 + (e & 7) * 16;
                    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4 *>(st + off) = z;
                    *reinterpret_cast<uint4 *>(st + kBlock + off) = z;
                    *reinterpret_cast<uint4 *>(st + kStageV + off) = z;
                    *reinterpret_cast<uint4 *>(st + kStageV + 8192 + off) = z;
                }
                fence_proxy_async();
            }
            if constexpr (kBf) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t part[3][16];
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float4 w4 = *reinterpret_cast<const float4 *>(w + hh * 32 + 2 * j);
                        const float ws[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int t = hh * 32 + 2 * j + 2 * e;
                            float a = wv(t, ws[2 * e]), b = wv(t + 1, ws[2 * e + 1]);
                            // the upper 16 bits are a bf16 by truncation; what is left is exact
                            part[0][j + e] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
                            a -= __uint_as_float(__float_as_uint(a) & 0xffff0000u);
                            b -= __uint_as_float(__float_as_uint(b) & 0xffff0000u);
                            if constexpr (NT == 3) {
                                part[1][j + e] = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
                                a -= __uint_as_float(__float_as_uint(a) & 0xffff0000u);
                                b -= __uint_as_float(__float_as_uint(b) & 0xffff0000u);
                            }
                            part[NT - 1][j + e] = H::pack2(a, b);
                        }
                    }
                    if (hh == 0 && it > 0 && !(ok = wait(ds_done, it - 1))) break;
                    if (hh == 0) fence_after_sync();
#pragma unroll
                    for (int m = 0; m < NT; ++m) tmem_st16(lane_base + tW + 32 * m + 16 * hh, part[m]);
                }
                if (!ok) break;
            } else {
                float x[64], m = 0.f, sc, inv;
#pragma unroll
                for (int t = 0; t < 64; t += 4) {
                    const float4 w4 = *reinterpret_cast<const float4 *>(w + t);
                    x[t] = wv(t, w4.x);
                    x[t + 1] = wv(t + 1, w4.y);
                    x[t + 2] = wv(t + 2, w4.z);
                    x[t + 3] = wv(t + 3, w4.w);
                    m = fmaxf(fmaxf(m, fmaxf(fabsf(x[t]), fabsf(x[t + 1]))), fmaxf(fabsf(x[t + 2]), fabsf(x[t + 3])));
                }
                half_scale(m, sc, inv);
                if (it > 0 && !(ok = wait(ds_done, it - 1))) break;
                fence_after_sync();
                winv[(it & 1) * 128 + i] = inv;
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float a = sc * x[hh * 32 + 2 * j], b = sc * x[hh * 32 + 2 * j + 1];
                        hi[j] = H::pack2(a, b);
                        const float2 r = Half16<__half>::unpack2(hi[j]);
                        lo[j] = H::pack2(a - r.x, b - r.y);
                    }
                    tmem_st16(lane_base + tW + 16 * hh, hi);
                    tmem_st16(lane_base + tW + 32 + 16 * hh, lo);
                }
            }
            tmem_wait_st();
            fence_before_sync();
            arrive(w_ready);
        }
    } else if (warp < 12) {
        // ============================ outputs ============================
        regs_dec<96>();
        if constexpr (kOut) {
            const int i = (warp - 8) * 32 + lane;  // value feature
            const uint32_t lane_base = tm + ((uint32_t)((warp - 8) * 32) << 16);
            const float *sinv = reinterpret_cast<const float *>(sm + oSInv);
            const float *pinv = reinterpret_cast<const float *>(sm + oPInv);
            Cursor k;
            k.start();
            for (int it = 0; k.next(p); ++it) {
                const int n = min(C, k.x.len - k.c * C);
                if (!(ok = wait_full(it)) || !(ok = wait(o_done, it))) break;
                fence_after_sync();
                const float *eb = reinterpret_cast<const float *>(sm + oGate + (it % NS) * kGate) + 64;
                const float si = kBf ? 1.f : sinv[(it & 1) * 128 + i];
                // two tokens' outputs of two neighbouring features a word: even
                // lanes keep the even tokens, odd lanes the odd ones
                uint32_t word[32];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    float o1[32], o2[32];
                    tmem_ld32(lane_base + tO1 + 32 * hh, o1);
                    tmem_ld32(lane_base + tO2 + 32 * hh, o2);
#pragma unroll
                    for (int t = 0; t < 32; t += 4) {
                        const float4 e4 = *reinterpret_cast<const float4 *>(eb + hh * 32 + t);
                        float4 p4 = make_float4(1.f, 1.f, 1.f, 1.f);
                        if constexpr (!kBf)
                            p4 = *reinterpret_cast<const float4 *>(pinv + (it & 1) * 64 + hh * 32 + t);
                        const float es[4] = {e4.x, e4.y, e4.z, e4.w}, ps[4] = {p4.x, p4.y, p4.z, p4.w};
                        float o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = kBf ? fmaf(es[e], o2[t + e], o1[t + e])
                                       : fmaf(es[e] * si, o2[t + e], ps[e] * o1[t + e]);
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float give = (lane & 1) ? o[e] : o[e + 1];
                            const float got = __shfl_xor_sync(0xffffffffu, give, 1);
                            word[hh * 16 + (t + e) / 2] = (lane & 1) ? H::pack2(got, o[e + 1]) : H::pack2(o[e], got);
                        }
                    }
                }
                fence_before_sync();
                arrive(o_free);
                arrive(&empty[it % NS]);
                if (i < dv) {
                    const long row = (long)Hv * dv;
                    E *dst = reinterpret_cast<E *>(p.out) + (k.x.tok0 + (long)k.c * C + (lane & 1)) * row +
                             (long)k.x.h * dv + (i & ~1);
#pragma unroll
                    for (int t = 0; t < 64; t += 2)
                        if (t + (lane & 1) < n) *reinterpret_cast<uint32_t *>(dst + t * row) = word[t / 2];
                }
            }
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
            if (lane == 0) {
                const uint32_t id_r = idesc_f16(128, 64, false, false, kBf);
                const uint32_t id_o1 = idesc_f16(128, 64, true, false, kBf);
                const uint32_t id_o2 = idesc_f16(128, 64, false, false, kBf);
                const uint32_t id_ds = idesc_f16(128, dk, false, true, kBf);
                const int ks = dk / 16;  // K = 16 steps over dk
                const uint32_t s0 = smem_u32(sm);
                auto w = [&](uint64_t *bar, int it) { return mbar_wait(bar, (uint32_t)it & 1u, p.wait_ns); };
                auto raw_scores = [&](int it) {
                    if (!w(&full[it % NS], it / NS) || (it > 0 && !w(r_free, it - 1))) return false;
                    fence_after_sync();
                    const uint32_t st = s0 + (it % NS) * kStage;
                    const uint64_t kq = desc_sw128(st, 16, 1024);
                    for (int k = 0; k < ks; ++k) {
                        const uint64_t d = desc_add(kq, (k >> 2) * kBlock + (k & 3) * 32);
                        mma_f16(tm + tR, d, d, id_r, k > 0);
                    }
                    mma_commit(r_done);
                    return true;
                };
                Cursor k;
                k.start();
                bool more = k.next(p);
                if constexpr (kOut) ok = !more || raw_scores(0);
                for (int it = 0; ok && more; ++it) {
                    const uint32_t st = s0 + (it % NS) * kStage;
                    // dS = W^T K, every part of W
                    if (!(ok = w(&full[it % NS], it / NS)) || !(ok = w(w_ready, it)) ||
                        (it > 0 && !(ok = w(ds_free, it - 1))))
                        break;
                    fence_after_sync();
                    const uint64_t kn = desc_sw128(st, kBlock, 1024);
#pragma unroll
                    for (int m = 0; m < NT; ++m)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma_f16_ta(tm + tDS, tm + tW + 32 * m + 8 * j, desc_add(kn, j * 2048), id_ds, m + j > 0);
                    mma_commit(ds_done);
                    if constexpr (kOut) {
                        // O2^T = S Q^T
                        if (!(ok = w(s_ready, it)) || (it > 0 && !(ok = w(o_free, it - 1)))) break;
                        fence_after_sync();
                        const uint64_t qd = desc_sw128(st + 8192, 16, 1024);
                        for (int j = 0; j < ks; ++j)
                            mma_f16_ta(tm + tO2, tm + tS + 8 * j, desc_add(qd, (j >> 2) * kBlock + (j & 3) * 32), id_o2,
                                       j > 0);
                        mma_commit(qs_done);
                        // O1^T = V^T P^T
                        if (!(ok = w(p_ready, it))) break;
                        fence_after_sync();
                        const uint64_t vd = desc_sw128(st + kStageV, 8192, 1024), pd = desc_sw128(s0 + oP, 16, 1024);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma_f16(tm + tO1, desc_add(vd, j * 2048), desc_add(pd, j * 32), id_o1, j > 0);
                        mma_commit(o_done);
                    }
                    mma_commit(&empty[it % NS]);
                    more = k.next(p);
                    if constexpr (kOut)
                        if (more && !(ok = raw_scores(it + 1))) break;
                }
                mma_commit(drain);  // nothing may be in flight when TMEM is given back
                mbar_wait(drain, 0, kDefaultWaitNs);
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
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
                    float x[64];
                    float m = 0.f, sc = 1.f;
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        float r[32];
                        tmem_ld32(lane_base + tR + 32 * hh, r);
#pragma unroll
                        for (int j = 0; j < 32; j += 4) {
                            const float4 b4 = *reinterpret_cast<const float4 *>(b + 32 * hh + j);
                            const float bs[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int t = 32 * hh + j + e;
                                x[t] = t <= i ? r[j + e] * p.scale * ex2_approx(bi - bs[e]) : 0.f;
                                if constexpr (!kBf) m = fmaxf(m, fabsf(x[t]));
                            }
                        }
                    }
                    fence_before_sync();
                    arrive(r_free);
                    if constexpr (!kBf) {
                        float inv;
                        half_scale(m, sc, inv);
                        pinv[(it & 1) * 64 + i] = inv;
                    }
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        uint32_t v[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            v[e] = kBf ? H::pack2(x[8 * q + 2 * e], x[8 * q + 2 * e + 1])
                                       : H::pack2(sc * x[8 * q + 2 * e], sc * x[8 * q + 2 * e + 1]);
                        *reinterpret_cast<uint4 *>(sm + oP + sw128_chunk(i, q)) = make_uint4(v[0], v[1], v[2], v[3]);
                    }
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
                        cudaStream_t stream) {
    p.G_run = g_run;
    const long units = (long)p.B * p.Hv * g_run, sms = sm_count_of_current_device();
    if (units == 0) return cudaSuccess;
    cudaError_t e = set_smem_once<linear_kernel<E, MODE>>((int)kSmem);
    if (e != cudaSuccess) return e;
    linear_kernel<E, MODE><<<(unsigned)(units < sms ? units : sms), kThreads, kSmem, stream>>>(p, mq, mk, mv);
    return cudaGetLastError();
}

template <typename E>
cudaError_t launch_e(const LinearParams &p, long total_T, cudaStream_t stream) {
    constexpr bool bf = Half16<E>::kBf16;
    CUtensorMap mq, mk, mv;
    memset(&mq, 0, sizeof(mq));
    memset(&mk, 0, sizeof(mk));
    memset(&mv, 0, sizeof(mv));
    if (total_T > 0 && (!encode_token_map(&mq, p.q, p.Hk, total_T, bf, p.dk) ||
                        !encode_token_map(&mk, p.k, p.Hk, total_T, bf, p.dk) ||
                        !encode_token_map(&mv, p.v, p.Hv, total_T, bf, p.dv)))
        return cudaErrorInvalidValue;
    if (p.G == 1) return launch_mode<E, kWhole>(p, 1, mq, mk, mv, stream);
    // the last segment's end state is only needed for the final state
    cudaError_t e = launch_mode<E, kStateOnly>(p, p.s_final != nullptr ? p.G : p.G - 1, mq, mk, mv, stream);
    if (e != cudaSuccess) return e;
    return launch_mode<E, kOutputs>(p, p.G, mq, mk, mv, stream);
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
