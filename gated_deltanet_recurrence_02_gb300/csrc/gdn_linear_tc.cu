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
// Precision.  The state stays in fp32 registers; sums of decays are fp32.  Roundings
// to 16 bits, and why each is enough:
//   W    is given to the MMAs as a sum of 16-bit parts.  bf16: w v in fp32, cut into
//        three parts of 8 bits, which is exact: the state is as good as one updated in
//        fp32.  Where only outputs read the state (the second pass over segments) two
//        parts, 2^-17, are below the outputs' rounding.  fp16: two parts, 22 bits,
//        scaled as below.
//   P, the state's image as an MMA operand: once each to the inputs' type, which is
//        the outputs' own rounding again.
// With fp16, W and the image are scaled per lane, and P per token, by powers of two, so
// neither small nor large states leave fp16's range.
//
// What bounds it.  A chunk and head of dk = dv = 128 moves 48 KB where two value heads
// share their keys and queries (2100 cycles of an SM's share of HBM bandwidth), and its
// products take about 1630 cycles of the tensor pipe (390 R, 195 O1, 260 O2, 780 dS:
// an M = 128, K = 16 MMA runs for 49 cycles at N = 64 with A in shared memory, 33 with A
// in TMEM, 65 at N = 128).  Measured: 64 packed rows of 500 to 1500 tokens, 32 heads,
// bf16: 343 us without initial states, 370 with (5.0 TB/s, 0.74 of the measured copy
// bandwidth), some 2100 cycles a chunk: between the end of one dS and the start of the
// next stand the state warps' read of it and, with one buffer of W, the store of the next
// W's first half, and every role's instructions compete for the issue slots and the
// instruction cache.  (A ring of W in blocks of 16 tokens, stored while the last product
// runs, gained nothing; nor did freeing the outputs' columns before their last part.)
// One row of 4100 tokens: 57 us, two passes of 25 and 31 us (a chunk takes a CTA as long
// alone, and 17 of them one after another are most of a pass).  12 rows of 200 to 1000
// tokens, 6 heads, d = 64, fp16: 33 to 35 us, the same chain.  128 rows of 16 tokens with their
// states: 161 us (0.54): a unit's state is read, used and written by the same four warps.
//
// One persistent CTA a SM, warp-specialised, four stages of tiles in flight; every
// hand-off between the roles is an mbarrier:
//   warps 0-3   state: dS -> fp32 registers -> the next chunk's image
//   warps 4-7, 20-23  W: values (ldmatrix, transposed), scaled and split, -> TMEM
//   warps 8-11  outputs: O1 + 2^{b} O2, transposed through shared memory (stmatrix), TMA stores
//   warp 12     tiles (TMA)
//   warp 13     issues dS
//   warps 14, 15, 19  P
//   warp 16     issues R, one chunk ahead, O2 and O1 (two issuing warps: an MMA costs
//               its issuer some 40 cycles, and half of them run for 33 to 49)
//   warps 17-18 the chunks' decay sums, up to eight chunks ahead
// What made the difference, at 64 packed rows: MMAs issued by a whole converged warp
// with descriptors at constant offsets, TMEM moved in fragment layouts and outputs by
// TMA, 1345 -> 433 us; code small enough for the instruction cache (each role's loops
// rolled where they can be), 433 -> 390 us; W formed in registers by two warpgroups and
// P on three warps, 390 -> 370 us; three parts of W for four, states prefetched, and W's
// loop rolled, 370 -> 343 us.  (Where a cold loop stands can cost as much: the tile warp's
// last waits, moved behind the roles or with another form of the wait, 343 -> 357 to 365.)
//
// Few rows are cut into segments of whole chunks, so that every SM has one: a
// first pass (kStateOnly) forms each segment's end state from zeros, a small kernel
// joins them along the row, and the second pass takes each segment's start state from
// those.  (Joining them in the second pass, by the state warps, took as long as its
// chunks: a thread is a row of the state there, and has few registers left.)
//
// Ragged chunks: tokens past the row's end get decay 1 and W = 0, and their K
// and V rows are zeroed in shared memory, so that nothing of the next row (NaN
// and infinities included) enters a product.
//
// Every wait is bounded; on timeout the CTA raises GDN_DEVERR_TIMEOUT, waits
// (bounded) for its copies and MMAs in flight, releases its TMEM and exits.
#include <algorithm>
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
constexpr int kThreads = 768;

// Shared memory: per stage two blocks (dk 0-63, 64-127) of [K 64 rows | Q 64
// rows] and two blocks of V; then P, the outputs, the stages' decay sums, the power-of-two
// scales (fp16) and the barriers.
constexpr uint32_t kBlock = 16384;
constexpr uint32_t kStageV = 2 * kBlock;
constexpr uint32_t kStage = kStageV + 16384;
constexpr uint32_t oP = NS * kStage;
constexpr uint32_t oOut = oP + 8192;               // [4 warps][64 tokens][32 features] on their way out
constexpr uint32_t oGate = oOut + 16384;           // kGates slots of kGate bytes, the words below
constexpr int kGates = 8;
constexpr uint32_t kGate = 912;
constexpr int gSum = 0;                            // [64] b_t, or b_t - b_31 from token 32 on (decays of at least 2^-127 each)
constexpr int gScaled = 64;                        // [64] scale 2^{b_t}
constexpr int gW = 128;                            // 2^{s_t}: fp32 [64], or bf16 [32 pairs][two parts]
constexpr int gLeft = 192;                         // [32] 2^{b_31 - b_t}
constexpr int gLast = 224;                         // 2^{b_63}
constexpr int gN = 225, gTok = 226, gHead = 227;   // ints: the chunk's tokens (0: no more chunks), first token, head
constexpr uint32_t oWExp = oGate + kGates * kGate; // [4][128] int8: the exponent of a lane's scale of W
constexpr uint32_t oSExp = oWExp + 512;            // [2][128] int8: of a lane's scale of the image
constexpr uint32_t oPInv = oSExp + 256;           // [2][64]  1 / scale of a row of P
constexpr uint32_t oPMax = oPInv + 512;            // [2][64] maxima of both parts of the later rows of P
constexpr uint32_t oBar = oPMax + 512;
constexpr uint32_t kSmem = oBar + 384 + 1024;      // + alignment slack

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
    uint32_t limit;    // of waits, ns: wait_ns, 4 s at most
    unsigned n_units;  // B Hv G_run
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

__device__ __forceinline__ uint32_t bf2_mul(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t bf2_fma(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
// a b - c: the rest of a product c = a b that was rounded to bf16, exactly.
__device__ __forceinline__ uint32_t bf2_rest(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("{\n\t.reg .b32 t;\n\tneg.bf16x2 t, %3;\n\tfma.rn.bf16x2 %0, %1, %2, t;\n}\n" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// The exponent of the power of two that brings a largest magnitude m into
// [2^13, 2^14) (fp16 holds 2^-14 .. 2^15 in full precision).
__device__ __forceinline__ int half_exp(float m) {
    const int e = 13 + 127 - (int)(__float_as_uint(m) >> 23);
    return !(m > 0.f) ? 0 : e > 126 ? 126 : e < -126 ? -126 : e;
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

// One unit: a segment of a (row, value head).
struct Unit {
    int b, h, g, len, c0, c1;
    long tok0;
};
__device__ __forceinline__ Unit unit_at(const LinearParams &p, unsigned u) {
    Unit x;
    const unsigned r = u / (unsigned)p.Hv;
    x.h = (int)(u - r * (unsigned)p.Hv);
    x.b = (int)(r / (unsigned)p.G_run);
    x.g = (int)(r - (unsigned)x.b * (unsigned)p.G_run);
    row_range(p.cu_seqlens, x.b, p.T, x.tok0, x.len);
    const unsigned nc = (unsigned)(x.len + C - 1) / C, per = (nc + p.G - 1) / (unsigned)p.G;
    x.c0 = (int)min((unsigned)x.g * per, nc);
    x.c1 = (int)min((unsigned)x.c0 + per, nc);
    return x;
}

template <typename E, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
linear_kernel(const LinearParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
              const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo) {
    using H = Half16<E>;
    constexpr bool kBf = H::kBf16;
    constexpr bool kOut = MODE != kStateOnly;
    constexpr int NT = kBf && MODE != kOutputs ? 3 : 2;  // 16-bit parts of W
    // Buffers of W and of dS in TMEM: two where the columns allow it, so that a
    // product need not wait for what reads or replaces the last one's.
    constexpr int WB = MODE == kStateOnly || NT == 2 ? 2 : 1, DB = MODE == kStateOnly ? 2 : 1;
    constexpr uint32_t cDS = MODE == kStateOnly ? 0 : tDS, cW = MODE == kStateOnly ? 256 : tW;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_align1k(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + oBar), *empty = full + NS;
    uint64_t *g_full = empty + NS, *g_empty = g_full + kGates;
    uint64_t *r_done = g_empty + kGates, *r_free = r_done + 1, *p_ready = r_done + 2, *qs_done = r_done + 3,
             *s_ready = r_done + 4, *o_done = r_done + 5, *o_free = r_done + 6, *drain = r_done + 7;
    // of even and of odd chunks, where a wait may lie more than one chunk back
    uint64_t *w_ready = r_done + 8, *ds_half = r_done + 10, *ds_done = r_done + 12, *ds_free = r_done + 14;
    uint64_t *max_there = r_done + 16;  // both parts' maxima of the later rows of P
    uint32_t *slot = reinterpret_cast<uint32_t *>(r_done + 17);
    // (through a shuffle: known to be the same in every lane)
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int dk = p.dk, dv = p.dv, Hv = p.Hv;

    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kOut ? 2 : 1);  // the warps that issue MMAs
        }
        for (int s = 0; s < kGates; ++s) {
            mbar_init(&g_full[s], 1);
            mbar_init(&g_empty[s], kOut ? 4 + 4 : 4);  // the last readers: state warps, output warps
        }
        mbar_init(r_done, 1);
        mbar_init(r_free, 3);
        mbar_init(p_ready, 3);
        mbar_init(max_there, 2);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&w_ready[s], 8);
            mbar_init(&ds_half[s], 1);
            mbar_init(&ds_done[s], 1);
            mbar_init(&ds_free[s], 4);
        }
        mbar_init(qs_done, 1);
        mbar_init(s_ready, 4);
        mbar_init(o_done, 1);
        mbar_init(o_free, 4);
        mbar_init(drain, kOut ? 2 : 1);
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
    if constexpr (MODE == kStateOnly) grid_launch_dependents();
    bool ok = true;
    // Waits run out p.limit nanoseconds after the warp's last chunk came.  (The roles'
    // loops share the instruction cache, and every wait's instructions count there:
    // 64 packed rows took 400 us with 3 KB more of them, 343 with 4 KB less.)
    uint32_t since = globaltimer_lo();
    // A wait of a whole warp: the outcome is the same in every lane, so that
    // the warp-wide TMEM accesses behind it stay converged.
    auto wait = [&](uint64_t *bar, int it) {
        return __all_sync(0xffffffffu, mbar_wait_since(bar, (uint32_t)it & 1u, since, p.limit)) != 0;
    };
    auto wait2 = [&](uint64_t *bars, int it) { return wait(&bars[it & 1], it >> 1); };
    auto gate_of = [&](int it) { return reinterpret_cast<float *>(sm + oGate + (it % kGates) * kGate); };
    // The chunk's decay sums are there; its tokens n, or 0 past the last one (and -1
    // where the wait ran out).
    auto chunk = [&](int it) {
        if (!wait(&g_full[it % kGates], it / kGates)) return -1;
        since = globaltimer_lo();
        return reinterpret_cast<const int *>(gate_of(it))[gN];
    };
    auto tiles = [&](int it) { return wait(&full[it % NS], it / NS); };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    if (warp < 4) {
        // ============================ state ==============================
        regs_inc<168>();
        const int i = warp * 32 + lane;  // value feature
        const uint32_t lane_base = tm + ((uint32_t)(warp * 32) << 16);
        const int8_t *wexp = reinterpret_cast<const int8_t *>(sm + oWExp);
        int8_t *sexp = reinterpret_cast<int8_t *>(sm + oSExp);
        float2 S[64];  // columns 2 j, 2 j + 1
        if constexpr (MODE == kOutputs) grid_dependency_wait();  // the fold's states
        int it = 0;
        const size_t mat = (size_t)dv * dk;
        // (a limit below a microsecond gives up where the first chunk is not there yet;
        // the other roles then wait for the state in vain)
        if (p.limit < 1000) ok = __all_sync(0xffffffffu, mbar_test_wait(&g_full[0], 0)) != 0;
#pragma unroll 1
        for (unsigned u = blockIdx.x; ok && u < p.n_units; u += gridDim.x) {
            const Unit x = unit_at(p, u);
            const size_t seg0 = ((size_t)x.b * Hv + x.h) * p.G;
            float *final = p.s_final != nullptr ? p.s_final + ((size_t)x.b * Hv + x.h) * mat : nullptr;
            // A last state in the place of the initial one: the unit of the row's first
            // segment copies it there in a second turn without chunks, when each thread
            // has read its row of the initial state.  (Else the fold has written it.)
            const int turns = MODE == kOutputs && x.g == 0 && final != nullptr && p.s_final == p.s0 ? 2 : 1;
#pragma unroll 1
            for (int turn = 0; ok && turn < turns; ++turn) {
                // the start: the initial state, or the state after the segment before
                const float *src = nullptr;
                if (x.g == 0 && turn == 0)
                    src = initial_state_ptr(p.s0, p.s0_idx, p.n_s0, x.b, x.h, Hv, dv, dk, p.err);
                else if (MODE == kOutputs)
                    src = p.seg_state + (seg0 + (turn == 0 ? x.g : p.G) - 1) * mat;
#pragma unroll
                for (int j = 0; j < 64; ++j) S[j] = make_float2(0.f, 0.f);
                if (src != nullptr && i < dv) {
                    src += (size_t)i * dk;
                    // (a lane is a row: 32-byte loads, as ld8_wide explains)
                    if ((reinterpret_cast<uintptr_t>(src) & 31) == 0) {
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            if (q * 8 < dk) ld8_wide(src + q * 8, S[4 * q], S[4 * q + 1], S[4 * q + 2], S[4 * q + 3]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 32; ++q)
                            if (q * 4 < dk) {
                                const float4 f = *reinterpret_cast<const float4 *>(src + q * 4);
                                S[2 * q] = make_float2(f.x, f.y);
                                S[2 * q + 1] = make_float2(f.z, f.w);
                            }
                    }
                }
                float kept = 1.f;  // the segment's decay
#pragma unroll 1
                for (int c = turn == 0 ? x.c0 : x.c1; c < x.c1; ++c, ++it) {
                    if constexpr (kOut) {
                        // this chunk's start state as an MMA operand
                        float sc = 1.f;
                        int se = 0;
                        if constexpr (!kBf) {
                            float m = 0.f;
#pragma unroll
                            for (int j = 0; j < 64; ++j) m = fmaxf(m, fmaxf(fabsf(S[j].x), fabsf(S[j].y)));
                            se = half_exp(m);
                            sc = pow2(se);
                        }
                        if (it > 0 && !(ok = wait(qs_done, it - 1))) break;
                        fence_after_sync();
                        // (the outputs two chunks back have read their scales: that
                        // product was issued after them)
                        if constexpr (!kBf) sexp[(it & 1) * 128 + i] = (int8_t)se;
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
                    if (!(ok = chunk(it) > 0) || !(ok = wait2(ds_done, it))) break;
                    fence_after_sync();
                    const float gam = gate_of(it)[gLast];
                    const float wi = kBf ? 1.f : pow2(-wexp[(it & 3) * 128 + i]);
                    const float2 gam2 = make_float2(gam, gam), wi2 = make_float2(wi, wi);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        if (g * 32 < dk) {
                            uint32_t v[32];
                            tmem_ld32_async(lane_base + cDS + 128 * (it % DB) + 32 * g, v);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                float2 d = make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1]));
                                if constexpr (!kBf) d = __fmul2_rn(wi2, d);
                                S[16 * g + j] = __ffma2_rn(gam2, S[16 * g + j], d);
                            }
                        }
                    }
                    kept *= gam;
                    fence_before_sync();
                    arrive(&ds_free[it & 1]);
                    arrive(&g_empty[it % kGates]);
                }
                if (!ok) break;
                float *dst = MODE == kWhole || turn == 1 ? final : nullptr;
                if (MODE == kStateOnly) {
                    dst = p.seg_state + (seg0 + x.g) * mat;
                    if (i == 0) p.seg_decay[seg0 + x.g] = kept;
                }
                if (dst != nullptr && i < dv) {
                    dst += (size_t)i * dk;
                    if ((reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
#pragma unroll
                        for (int q = 0; q < 16; ++q)
                            if (q * 8 < dk) st8_wide(dst + q * 8, S[4 * q], S[4 * q + 1], S[4 * q + 2], S[4 * q + 3]);
                    } else {
#pragma unroll
                        for (int q = 0; q < 32; ++q)
                            if (q * 4 < dk)
                                *reinterpret_cast<float4 *>(dst + q * 4) =
                                    make_float4(S[2 * q].x, S[2 * q].y, S[2 * q + 1].x, S[2 * q + 1].y);
                    }
                }
            }
        }
    } else if (warp < 8 || warp >= 20) {
        // ============================== W ================================
        // Two warps for each 32 features, 16 of them each.
        regs_dec<64>();
        const int wq = warp & 3, hh = warp >= 20 ? 1 : 0;
        const uint32_t lane_base = tm + ((uint32_t)(wq * 32 + 16 * hh) << 16);
        int8_t *wexp = reinterpret_cast<int8_t *>(sm + oWExp) + wq * 32 + 16 * hh + (lane >> 2);
        // ldmatrix: this lane's row of the four 8 x 8 matrices (tokens 0-7 and
        // 8-15 of 16, features 0-7 and 8-15 of 16)
        const int row = (lane & 7) + ((lane >> 4) << 3), cg = (wq & 1) * 4 + 2 * hh + ((lane >> 3) & 1);
        const uint32_t v_off = kStageV + (wq >> 1) * 8192 + row * 128 + ((cg ^ (lane & 7)) << 4);
#pragma unroll 1
        for (int it = 0;; ++it) {
            const int n = chunk(it);
            ok = n >= 0;
            if (n <= 0) break;
            if (!(ok = tiles(it))) break;
            uint8_t *st = sm + (it % NS) * kStage;
            if (n < C) {
                // Rows past the row's end: zeros, whatever was loaded.  Of V this warp's own
                // 16 features, which no other warp reads for W; of K an eighth, which the
                // product reads behind all eight warps' w_ready.  (So no barrier stands
                // here, which a warp whose wait ran out would leave the others in.)
                const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
                for (int e = (wq + 4 * hh) * 32 + lane; e < (C - n) * 8; e += 256) {
                    const int off = (n + (e >> 3)) * 128 + (e & 7) * 16;
                    *reinterpret_cast<uint4 *>(st + off) = z;
                    *reinterpret_cast<uint4 *>(st + kBlock + off) = z;
                }
#pragma unroll 1
                for (int e = lane; e < (C - n) * 2; e += 32)
                    *reinterpret_cast<uint4 *>(st + kStageV + (wq >> 1) * 8192 +
                                               sw128_chunk(n + (e >> 1), (wq & 1) * 4 + 2 * hh + (e & 1))) = z;
                fence_proxy_async();
                __syncwarp();
            }
            // 16 tokens (j): features g and g + 8, tokens 2 t, 2 t + 1 of each eight,
            // which is the layout of the TMEM store
            auto values = [&](int j, uint32_t (&v)[4]) { ldsm_x4_trans(v, st + v_off + j * 2048); };
            float sc[2] = {1.f, 1.f};
            int we[2];
            auto scaled = [&](int j, float2 (&x)[4]) {  // fp16: in fp32
                uint32_t v[4];
                values(j, v);
                const float *w = gate_of(it) + gW + 2 * (lane & 3) + 16 * j;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    x[e] = __fmul2_rn(*reinterpret_cast<const float2 *>(w + 8 * (e >> 1)), H::unpack2(v[e]));
            };
            if constexpr (!kBf) {
                // the largest magnitude of each feature gives its scale; the four
                // lanes of a group hold a feature's tokens
                float m[2] = {0.f, 0.f};
#pragma unroll 1
                for (int j = 0; j < 4; ++j) {
                    float2 x[4];
                    scaled(j, x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) m[e & 1] = fmaxf(m[e & 1], fmaxf(fabsf(x[e].x), fabsf(x[e].y)));
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], 1));
                    m[e] = fmaxf(m[e], __shfl_xor_sync(0xffffffffu, m[e], 2));
                    we[e] = half_exp(m[e]);
                    sc[e] = pow2(we[e]);
                }
            }
            // 16 tokens at a time.  Each half of the chunk is formed while the last
            // chunk's product still reads that half of TMEM.
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                uint32_t part[NT][4];
                if constexpr (kBf && NT == 2) {
                    // packed bf16 arithmetic: with w = w0 + w1 to 16 bits, w0 v is
                    // exactly its rounding plus a rest
                    uint32_t v[4];
                    values(j, v);
                    const uint2 *w = reinterpret_cast<const uint2 *>(gate_of(it) + gW) + (lane & 3) + 8 * j;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint2 ww = w[4 * (e >> 1)];
                        const uint32_t a = bf2_mul(ww.x, v[e]);
                        part[0][e] = a;
                        part[1][e] = bf2_fma(ww.y, v[e], bf2_rest(ww.x, v[e], a));
                    }
                } else if constexpr (kBf) {
                    // w v in fp32, cut into its bits 0-7, 8-15 and 16-23
                    float2 x[4];
                    scaled(j, x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
#pragma unroll
                        for (int m = 0; m < 3; ++m) {
                            const uint32_t a = __float_as_uint(x[e].x), b = __float_as_uint(x[e].y);
                            part[m][e] = __byte_perm(a, b, 0x7632);
                            if (m < 2)
                                x[e] = __ffma2_rn(make_float2(-1.f, -1.f),
                                                  make_float2(__uint_as_float(a & 0xffff0000u),
                                                              __uint_as_float(b & 0xffff0000u)),
                                                  x[e]);
                        }
                    }
                } else {
                    float2 x[4];
                    scaled(j, x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 r = __fmul2_rn(make_float2(sc[e & 1], sc[e & 1]), x[e]);
                        part[0][e] = H::pack2(r.x, r.y);
                        const float2 h = H::unpack2(part[0][e]);
                        part[1][e] = H::pack2(r.x - h.x, r.y - h.y);
                    }
                }
                if (it >= WB && (j & 1) == 0 && !(ok = wait2(j == 0 ? ds_half : ds_done, it - WB))) break;
                fence_after_sync();
#pragma unroll
                for (int m = 0; m < NT; ++m) tmem_st_16x8(lane_base + cW + 32 * NT * (it % WB) + 32 * m + 8 * j, part[m]);
            }
            if (!ok) break;
            // (four buffers: the state warps read their scale before the product two
            // chunks on, whose end was waited for two chunks after that at the latest)
            if constexpr (!kBf)
                if ((lane & 3) == 0)
#pragma unroll
                    for (int e = 0; e < 2; ++e) wexp[(it & 3) * 128 + 8 * e] = (int8_t)we[e];
            tmem_wait_st();
            fence_before_sync();
            arrive(&w_ready[it & 1]);
        }
        if (!ok) tmem_wait_st();  // given up between two halves: TMEM is freed behind the stores
    } else if (warp < 12) {
        // ============================ outputs ============================
        regs_dec<64>();
        if constexpr (kOut) {
            const int wq = warp - 8;
            const uint32_t lane_base = tm + ((uint32_t)(wq * 32) << 16);
            const int8_t *sexp = reinterpret_cast<const int8_t *>(sm + oSExp) + wq * 32 + (lane >> 2);
            const float *pinv = reinterpret_cast<const float *>(sm + oPInv) + 2 * (lane & 3);
            uint8_t *buf = sm + oOut + wq * 4096;  // [64 tokens][32 features], 64-byte swizzle
            // stmatrix: this lane's row (token) of the four 8 x 8 matrices (features
            // 0-7 and 8-15 of 16, tokens 0-7 and 8-15 of 16)
            const int row = (lane & 7) + ((lane >> 4) << 3), cg = (lane >> 3) & 1;
#pragma unroll 1
            for (int it = 0;; ++it) {
                const int n = chunk(it);
                ok = n >= 0;
                if (n <= 0 || !(ok = wait(o_done, it))) break;
                fence_after_sync();
                const float *eb = gate_of(it) + gScaled + 2 * (lane & 3);
                const int t0 = reinterpret_cast<const int *>(gate_of(it))[gTok];
                const int h = reinterpret_cast<const int *>(gate_of(it))[gHead];
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
                                const float si = pow2(-sexp[(it & 1) * 128 + 16 * hh + 8 * m]);
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
                arrive(&g_empty[it % kGates]);
                if (wq * 32 >= dv) continue;
                if (n == C) {
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_3d(&mo, wq * 32, h, t0, buf);
                        bulk_commit();
                    }
                } else {  // the next row's tokens stay untouched
                    __syncwarp();
#pragma unroll 1
                    for (int e = lane; e < n * 4; e += 32) {
                        const int t = e >> 2, q = e & 3;
                        *reinterpret_cast<uint4 *>(reinterpret_cast<E *>(p.out) + ((long)(t0 + t) * Hv + h) * dv + wq * 32 + 8 * q) =
                            *reinterpret_cast<const uint4 *>(buf + t * 64 + ((q ^ ((t >> 1) & 3)) << 4));
                    }
                    __syncwarp();
                }
            }
            if (lane == 0) bulk_wait_all();
        }
    } else if (warp < 16) {
        regs_dec<72>();
        const uint32_t leader = elect_leader();
        if (warp == 12) {
            // ============================ tiles ==========================
            const int G = Hv / p.Hk, bytes = 8192 * ((dk > 64 ? 2 : 1) * (kOut ? 2 : 1) + (dv > 64 ? 2 : 1));
            unsigned u = blockIdx.x;
            int it = 0;
#pragma unroll 1
            for (; ok && u < p.n_units; u += gridDim.x) {
                const Unit x = unit_at(p, u);
                const int hk = x.h / G;
                // The unit's initial state to L2, up to four chunks before the state warps
                // read it: 64 packed rows with states 410 -> 392 us.  (Not for units of a
                // chunk or two, whose tiles it would hold up: 128 rows of 64 tokens 172 us,
                // 185 with it.)
                if (x.g == 0 && x.c1 - x.c0 > 2 && u != blockIdx.x) {
                    const float *s0 = initial_state_ptr(p.s0, p.s0_idx, p.n_s0, x.b, x.h, Hv, dv, dk, p.err);
                    if (s0 != nullptr && leader) bulk_prefetch_l2(s0, (uint32_t)(dv * dk) * 4);
                }
#pragma unroll 1
                for (int c = x.c0; c < x.c1; ++c, ++it) {
                    const int s = it % NS, t0 = (int)(x.tok0 + (long)c * C);
                    if (it >= NS && !(ok = wait(&empty[s], it / NS - 1))) break;
                    since = globaltimer_lo();
                    uint8_t *st = sm + s * kStage;
                    if (leader) mbar_arrive_expect_tx(&full[s], bytes);
                    __syncwarp();
#pragma unroll 1
                    for (int j = 0; j < 2; ++j) {
                        if (64 * j < dk) {
                            tma_load_3d_warp(leader, st + j * kBlock, &mk, 64 * j, hk, t0, &full[s]);
                            if constexpr (kOut) tma_load_3d_warp(leader, st + j * kBlock + 8192, &mq, 64 * j, hk, t0, &full[s]);
                        }
                        if (64 * j < dv) tma_load_3d_warp(leader, st + kStageV + j * 8192, &mv, 64 * j, x.h, t0, &full[s]);
                    }
                }
            }
            // The copies in flight must land before the CTA ends: the warps that read
            // the last tiles may have given up although this one did not.
#pragma unroll 1
            for (int j = it > NS ? it - NS : 0; j < it; ++j)
                mbar_wait(&full[j % NS], (uint32_t)(j / NS) & 1u, kDefaultWaitNs / 8);
        } else if (warp == 13) {
            // ================= MMAs of the state's update ================
            const uint32_t id_ds = idesc_f16(128, dk, false, true, kBf);
#pragma unroll 1
            for (int it = 0;; ++it) {
                const int n = chunk(it);
                ok = n >= 0;
                if (n <= 0) break;
                if (!(ok = tiles(it))) break;
                const uint32_t st = smem_u32(sm) + (it % NS) * kStage;
                // dS = W^T K, every part of 16 tokens of W at a time
                if (!(ok = wait2(w_ready, it)) || (it >= DB && !(ok = wait2(ds_free, it - DB)))) break;
                fence_after_sync();
                const uint64_t kn = desc_sw128(st, kBlock, 1024);
                const uint32_t ds = tm + cDS + 128 * (it % DB), w = tm + cW + 32 * NT * (it % WB);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
#pragma unroll
                    for (int m = 0; m < NT; ++m)
                        mma_f16_ta_warp(leader, ds, w + 32 * m + 8 * j, desc_add(kn, j * 2048), id_ds, m + j > 0);
                    if (j == 1) mma_commit_warp(leader, &ds_half[it & 1]);
                }
                mma_commit_warp(leader, &ds_done[it & 1]);
                mma_commit_warp(leader, &empty[it % NS]);
            }
            mma_commit_warp(leader, drain);  // nothing may be in flight when TMEM is given back
            mbar_wait(drain, 0, kDefaultWaitNs);
        } else if constexpr (kOut) {
            // ============ P: the rows' diagonal blocks of 32 columns ==========
            const int diag = 32 * (warp - 14);
            const int i = diag + lane;  // token of the chunk
            const uint32_t lane_base = tm + ((uint32_t)(64 + diag) << 16);
            float *pinv = reinterpret_cast<float *>(sm + oPInv);
            const float2 scale2 = make_float2(p.scale, p.scale);
            if (diag == 0)  // right of the first rows' block: zeros, once
#pragma unroll 1
                for (int q = 4; q < 8; ++q)
                    *reinterpret_cast<uint4 *>(sm + oP + sw128_chunk(i, q)) = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 1
            for (int it = 0;; ++it) {
                const int n = chunk(it);
                ok = n >= 0;
                if (n <= 0 || !(ok = wait(r_done, it))) break;
                fence_after_sync();
                uint32_t x[32];
                tmem_ld32_async(lane_base + tR + diag, x);
                tmem_wait_ld();
                fence_before_sync();
                arrive(r_free);
                if (n < C) {  // V rows past the row's end: zeros, whatever was loaded
                    uint8_t *v = sm + (it % NS) * kStage + kStageV;
#pragma unroll 1
                    for (int e = i; e < (C - n) * 8; e += 64) {
                        const int off = (n + (e >> 3)) * 128 + (e & 7) * 16;
                        *reinterpret_cast<uint4 *>(v + off) = make_uint4(0u, 0u, 0u, 0u);
                        *reinterpret_cast<uint4 *>(v + 8192 + off) = make_uint4(0u, 0u, 0u, 0u);
                    }
                }
                const float *b = gate_of(it) + gSum + diag;
                const float bi = b[lane];
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < 32; j += 2) {
                    const float2 b2 = *reinterpret_cast<const float2 *>(b + j);
                    float2 v = make_float2(__uint_as_float(x[j]), __uint_as_float(x[j + 1]));
                    v = __fmul2_rn(__fmul2_rn(v, scale2), make_float2(ex2_approx(bi - b2.x), ex2_approx(bi - b2.y)));
                    v.x = j <= lane ? v.x : 0.f;
                    v.y = j + 1 <= lane ? v.y : 0.f;
                    if constexpr (kBf) {
                        x[j / 2] = H::pack2(v.x, v.y);
                    } else {
                        m = fmaxf(m, fmaxf(fabsf(v.x), fabsf(v.y)));
                        x[j] = __float_as_uint(v.x);
                        x[j + 1] = __float_as_uint(v.y);
                    }
                }
                // the products with the last chunk's P are done (and so are the reads
                // of the scales of the one before)
                if (it > 0 && !(ok = wait(o_done, it - 1))) break;
                if constexpr (!kBf) {
                    if (diag > 0) {  // one scale a row: with the maximum of its left part
                        float *pmax = reinterpret_cast<float *>(sm + oPMax) + (it & 1) * 64;
                        pmax[lane] = m;
                        arrive(max_there);
                        if (!(ok = wait(max_there, it))) break;
                        m = fmaxf(m, pmax[32 + lane]);
                    }
                    const int pe = half_exp(m);
                    const float sc = pow2(pe);
                    pinv[(it & 1) * 64 + i] = pow2(-pe);
#pragma unroll
                    for (int j = 0; j < 32; j += 2)
                        x[j / 2] = H::pack2(sc * __uint_as_float(x[j]), sc * __uint_as_float(x[j + 1]));
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<uint4 *>(sm + oP + sw128_chunk(i, diag / 8 + q)) =
                        make_uint4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
                fence_proxy_async();
                arrive(p_ready);
            }
        }
    } else {
        regs_dec<48>();
        const uint32_t leader = elect_leader();
        if (warp == 16) {
            // ===================== MMAs of the outputs ===================
            if constexpr (kOut) {
                const uint32_t id_r = idesc_f16(128, 64, false, false, kBf);
                const uint32_t id_o1 = idesc_f16(128, 64, true, false, kBf);
                const uint32_t s0 = smem_u32(sm);
                // K = 16 steps over dk, each with constant offsets: an MMA whose
                // descriptor is computed in a loop costs its issuer twice the time
                auto over_dk = [&](auto step) {
                    step(0);
                    step(1);
                    if (dk >= 64) {
                        step(2);
                        step(3);
                    }
                    if (dk == 128) {
                        step(4);
                        step(5);
                        step(6);
                        step(7);
                    }
                };
#pragma unroll 1
                for (int it = 0;; ++it) {
                    const int n = chunk(it);
                    ok = n >= 0;
                    if (n > 0) {
                        // R = [K;Q] K^T
                        if (!(ok = tiles(it)) || (it > 0 && !(ok = wait(r_free, it - 1)))) break;
                        fence_after_sync();
                        const uint64_t kq = desc_sw128(s0 + (it % NS) * kStage, 16, 1024);
                        over_dk([&](int k) {
                            const uint64_t d = desc_add(kq, (k >> 2) * kBlock + (k & 3) * 32);
                            mma_f16_warp(leader, tm + tR, d, d, id_r, k > 0);
                        });
                        mma_commit_warp(leader, r_done);
                    }
                    if (it > 0 && ok) {
                        // of the chunk before: O2^T = S Q^T,
                        const int pt = it - 1;
                        if (!(ok = wait(s_ready, pt)) || (pt > 0 && !(ok = wait(o_free, pt - 1)))) break;
                        fence_after_sync();
                        const uint64_t qd = desc_sw128(s0 + (pt % NS) * kStage + 8192, 16, 1024);
                        over_dk([&](int k) {
                            mma_f16_ta_warp(leader, tm + tO2, tm + tS + 8 * k,
                                            desc_add(qd, (k >> 2) * kBlock + (k & 3) * 32), id_r, k > 0);
                        });
                        mma_commit_warp(leader, qs_done);
                        // and O1^T = V^T P^T
                        if (!(ok = wait(p_ready, pt))) break;
                        fence_after_sync();
                        const uint64_t vd = desc_sw128(s0 + (pt % NS) * kStage + kStageV, 8192, 1024);
                        const uint64_t pd = desc_sw128(s0 + oP, 16, 1024);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            mma_f16_warp(leader, tm + tO1, desc_add(vd, j * 2048), desc_add(pd, j * 32), id_o1, j > 0);
                        mma_commit_warp(leader, o_done);
                        mma_commit_warp(leader, &empty[pt % NS]);
                    }
                    if (n <= 0) break;
                }
                mma_commit_warp(leader, drain);
                mbar_wait(drain, 0, kDefaultWaitNs);
            }
        } else if (warp == 19) {
            if constexpr (kOut) {
                // ======== P: the columns left of the second diagonal block ========
                // 2^{b_i - b_31} 2^{b_31 - b_j}: two factors of at most 1 where no
                // decay is above 1.
                const int i = 32 + lane;  // token of the chunk
                const uint32_t lane_base = tm + (96u << 16);
#pragma unroll 1
                for (int it = 0;; ++it) {
                    const int n = chunk(it);
                    ok = n >= 0;
                    if (n <= 0 || !(ok = wait(r_done, it))) break;
                    fence_after_sync();
                    const float *gate = gate_of(it);
                    const float l = p.scale * ex2_approx(gate[gSum + i]);
                    float2 l2 = make_float2(l, l);
                    if constexpr (!kBf) {
                        float m = 0.f;
#pragma unroll 1
                        for (int hh = 0; hh < 2; ++hh) {
                            uint32_t y[16];
                            tmem_ld16_async(lane_base + tR + 16 * hh, y);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                m = fmaxf(m, fabsf(__uint_as_float(y[j]) * gate[gLeft + 16 * hh + j] * l));
                        }
                        // (two buffers: the next chunk's maxima may be there before the
                        // other warp has read these, the one after next's are not)
                        float *pmax = reinterpret_cast<float *>(sm + oPMax) + (it & 1) * 64;
                        pmax[32 + lane] = m;
                        arrive(max_there);
                        if (!(ok = wait(max_there, it))) break;
                        const float sc = pow2(half_exp(fmaxf(m, pmax[lane])));
                        l2 = make_float2(l * sc, l * sc);
                    }
                    if (it > 0 && !(ok = wait(o_done, it - 1))) break;
#pragma unroll 1
                    for (int hh = 0; hh < 2; ++hh) {
                        uint32_t y[16];
                        tmem_ld16_async(lane_base + tR + 16 * hh, y);
                        tmem_wait_ld();
                        if (hh == 1) {
                            fence_before_sync();
                            arrive(r_free);
                        }
#pragma unroll
                        for (int j = 0; j < 16; j += 2) {
                            const float2 c2 = *reinterpret_cast<const float2 *>(gate + gLeft + 16 * hh + j);
                            const float2 v =
                                __fmul2_rn(__fmul2_rn(make_float2(__uint_as_float(y[j]), __uint_as_float(y[j + 1])), c2), l2);
                            y[j / 2] = H::pack2(v.x, v.y);
                        }
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            *reinterpret_cast<uint4 *>(sm + oP + sw128_chunk(i, 2 * hh + q)) =
                                make_uint4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
                    }
                    fence_proxy_async();
                    arrive(p_ready);
                }
            }
        } else {
            // ========================= decay sums ========================
            // Two warps take the chunks in turn: a chunk's decays are loaded while
            // the warp's last one is worked on, and take longer than a chunk does.
            const bool per_head = (p.conv & GDN_ALPHA_PER_HEAD) != 0;
            unsigned u = blockIdx.x - gridDim.x;  // (wraps to blockIdx.x at the first step)
            Unit x;
            x.c1 = 0;
            int c = 0, t0 = 0, n = 0, h = 0;  // the chunk that is next: first token, tokens, head
            float raw[2] = {0.f, 0.f};        // its decays of tokens 2 lane, 2 lane + 1, as stored
            int steps = warp - 16;            // to the warp's next chunk
            bool end = false;                 // the next one would be the first past the last
            bool over = false;                // no more chunks
#pragma unroll 1
            for (int it = warp - 19;; it += 2) {
                const int t0_ = t0, n_ = n, h_ = h;
                const bool end_ = end;
                float a[2] = {raw[0], raw[1]};
                n = 0;
#pragma unroll 1
                for (; steps > 0 && !over; --steps) {
                    ++c;
#pragma unroll 1
                    while (c >= x.c1) {
                        u += gridDim.x;
                        if ((over = u >= p.n_units)) break;
                        x = unit_at(p, u);
                        c = x.c0;
                    }
                    end = over && steps == 1;
                }
                steps = 2;
                if (!over) {
                    t0 = (int)(x.tok0 + (long)c * C);
                    n = min(C, x.len - c * C);
                    h = x.h;
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        if (2 * lane + e < n)
                            raw[e] = ld_gate_early(p.alpha, per_head ? (long)h : (long)(t0 + 2 * lane + e) * Hv + h, p.dt_gate);
                }
                if (it < 0) continue;
                if (n_ == 0 && !end_) break;
                if (it >= kGates && !(ok = wait(&g_empty[it % kGates], it / kGates - 1))) break;
                since = globaltimer_lo();
                float *gate = gate_of(it);
                if (lane == 0) {
                    reinterpret_cast<int *>(gate)[gN] = n_;
                    reinterpret_cast<int *>(gate)[gTok] = t0_;
                    reinterpret_cast<int *>(gate)[gHead] = h_;
                }
                // Inclusive sums over the lanes from both ends; the exclusive ones
                // are the neighbours' (a difference would lose what a strong decay
                // has in front of it, and be no number after a decay of 0).  For
                // P's differences the sums start anew at token 32, and a decay below
                // 2^-127 (0 among them) counts as 2^-127: P's exponential of a difference
                // across it is 0 all the same, and the sums stay finite.  They are exact
                // to 2^-17 for decays that sum to less than 2^6 in a half, to 2^-13 a sum
                // for the strongest ones.
                float held[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    a[e] = 2 * lane + e >= n_ ? 0.f : (p.conv & GDN_ALPHA_LOG) ? a[e] * kLog2e : log2f(a[e]);
                    held[e] = a[e] < -127.f ? -127.f : a[e];
                }
                float up = a[0] + a[1], down = up, hup = held[0] + held[1];
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const float y0 = __shfl_up_sync(0xffffffffu, up, o), y1 = __shfl_down_sync(0xffffffffu, down, o);
                    const float y2 = __shfl_up_sync(0xffffffffu, hup, o);
                    if (lane >= o) up += y0;
                    if ((lane & 15) >= o) hup += y2;
                    if (lane + o < 32) down += y1;
                }
                float ex = __shfl_up_sync(0xffffffffu, up, 1), eh = __shfl_up_sync(0xffffffffu, hup, 1);
                float suf = __shfl_down_sync(0xffffffffu, down, 1);
                if (lane == 0) ex = 0.f;
                if ((lane & 15) == 0) eh = 0.f;
                if (lane == 31) suf = 0.f;
                const float b31 = __shfl_sync(0xffffffffu, hup, 15);
                const float2 b2 = make_float2(eh + held[0], hup);
                *reinterpret_cast<float2 *>(gate + gSum + 2 * lane) = b2;
                *reinterpret_cast<float2 *>(gate + gScaled + 2 * lane) =
                    make_float2(p.scale * ex2_approx(ex + a[0]), p.scale * ex2_approx(up));
                const float2 w2 = make_float2(ex2_approx(suf + a[1]), ex2_approx(suf));
                if constexpr (kBf && NT == 2) {
                    const uint32_t wa = H::pack2(w2.x, w2.y);
                    const float2 r = H::unpack2(wa);
                    *reinterpret_cast<uint2 *>(gate + gW + 2 * lane) = make_uint2(wa, H::pack2(w2.x - r.x, w2.y - r.y));
                } else {
                    *reinterpret_cast<float2 *>(gate + gW + 2 * lane) = w2;
                }
                if (lane < 16)
                    *reinterpret_cast<float2 *>(gate + gLeft + 2 * lane) =
                        make_float2(ex2_approx(b31 - b2.x), ex2_approx(b31 - b2.y));
                if (lane == 31) gate[gLast] = ex2_approx(up);
                arrive(&g_full[it % kGates]);
                if (n_ == 0) break;  // past the last chunk
            }
        }
    }
    if (!ok && lane == 0) atomicOr(p.err, (uint32_t)GDN_DEVERR_TIMEOUT);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 0) tmem_dealloc(tm, kTmemCols);
}

// Between the two passes: every segment's end state from the ones from zeros, in
// place, E_g <- decay_g E_{g-1} + E_g, and the row's last one to final (unless that
// is the initial state, which the second pass still reads).  Four columns a thread.
__global__ void __launch_bounds__(256) fold_kernel(const LinearParams p, float *final) {
    grid_launch_dependents();
    grid_dependency_wait();
    const size_t mat = (size_t)p.dv * p.dk, per = mat / 4;
    const size_t e = (size_t)blockIdx.x * 256 + threadIdx.x;
    const size_t bh = e / per, at = (e - bh * per) * 4;
    if (bh >= (size_t)p.B * p.Hv) return;
    float *m = p.seg_state + bh * p.G * mat + at;
    float4 run = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int g = 0; g < p.G_run; ++g) {
        const float d = p.seg_decay[bh * p.G + g];
        const float4 x = *reinterpret_cast<const float4 *>(m + g * mat);
        run = g == 0 ? x : make_float4(fmaf(d, run.x, x.x), fmaf(d, run.y, x.y), fmaf(d, run.z, x.z), fmaf(d, run.w, x.w));
        *reinterpret_cast<float4 *>(m + g * mat) = run;
    }
    if (final != nullptr) *reinterpret_cast<float4 *>(final + bh * mat + at) = run;
}

// Segments a row.  One pass takes its chunks one after another; two passes over G
// segments take each chunk of a segment twice (measured: 1.5 times one pass's time), as
// much as 8 chunks for the second launch, the fold and the states' way between them, and
// a third of a chunk a segment in the fold.  The least of these, with no more segments
// than one wave of SMs: 32 heads, 4100 tokens (65 chunks): 93 us as one segment, 84, 67
// and 61 us as 2, 3 and 4; 8 heads: 91 us, 51 as 4, 39 as 8, 43 as 19; but 64 heads,
// 2048 tokens: 54 us, 59 as 2, and 32 heads, 512 tokens: 23 us, 28 as 4.
int segments(int B, int T, int Hv, bool varlen) {
    const long sms = sm_count_of_current_device(), units = (long)B * Hv;
    if (units == 0) return 1;
    const long longest = varlen ? (T + B - 1) / B : T;  // packed rows: their mean
    const long chunks = (longest + C - 1) / C;
    long best = 6 * chunks;
    int G = 1;
    for (long g = 2; g <= sms / units && g <= chunks; ++g) {
        const long cost = 9 * ((chunks + g - 1) / g) + 48 + 2 * g;
        if (cost < best) {
            best = cost;
            G = (int)g;
        }
    }
    return G;
}

// A launch that may start while the one before it in the stream still runs.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), unsigned grid, int threads, uint32_t smem, cudaStream_t stream, bool early,
                         const A &...args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename E, int MODE>
cudaError_t launch_mode(LinearParams p, int g_run, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                        const CUtensorMap &mo, cudaStream_t stream) {
    p.G_run = g_run;
    const long units = (long)p.B * p.Hv * g_run, sms = sm_count_of_current_device();
    if (units == 0) return cudaSuccess;
    if (units > 0x7fffffffL - sms) return cudaErrorInvalidValue;
    p.n_units = (unsigned)units;
    cudaError_t e = set_smem_once<linear_kernel<E, MODE>>((int)kSmem);
    if (e != cudaSuccess) return e;
    // the second pass starts as SMs come free, and waits for the fold only where it
    // reads the states
    return launch_after(linear_kernel<E, MODE>, (unsigned)(units < sms ? units : sms), kThreads, kSmem, stream,
                        MODE == kOutputs, p, mq, mk, mv, mo);
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
    const int g_run = p.s_final != nullptr ? p.G : p.G - 1;
    cudaError_t e = launch_mode<E, kStateOnly>(p, g_run, mq, mk, mv, mo, stream);
    if (e != cudaSuccess) return e;
    LinearParams f = p;
    f.G_run = g_run;
    const size_t threads = (size_t)p.B * p.Hv * p.dv * p.dk / 4;
    e = launch_after(fold_kernel, (unsigned)((threads + 255) / 256), 256, 0, stream, true, f,
                     p.s_final != p.s0 ? p.s_final : nullptr);
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
    p.limit = (uint32_t)std::min<uint64_t>(p.wait_ns, 4000000000ull);
    if (p.G > 1) {
        p.seg_state = reinterpret_cast<float *>(p.ws);
        p.seg_decay = reinterpret_cast<float *>(static_cast<uint8_t *>(p.ws) + state_bytes(p.B, p.Hv, p.G, p.dk, p.dv));
    }
    return p.dt_qkv == GDN_BF16 ? launch_e<__nv_bfloat16>(p, total_T, stream) : launch_e<__half>(p, total_T, stream);
}

}  // namespace gdn
