// gdn_attention_tc.cu -- attention over a paged cache on the 5th-generation tensor cores
// (tcgen05 MMA, TMEM, TMA), for 16-bit tensors.
//
// Per query row, over tiles of 128 keys (x: raw scores, c = scale log2 e):
//     S = Q K^T,  m' = max(m, max_j S_j),  P_j = 2^{c S_j - c m'}
//     l <- 2^{c (m - m')} l + sum_j P_j,   O <- 2^{c (m - m')} O + P V
// and O / l at the end.  S and O are fp32 in TMEM, a query row to a lane, so a thread has a
// whole row of a tile: no reduction crosses threads.  m follows the true maximum only when
// that has grown by more than 8 in the exponent (running maximum and sum: M. Milakov and
// N. Gimelshein, "Online normalizer calculation for softmax" (2018); that the maximum may lag
// is known from published attention kernels): weights of up to 2^8 are as exact, and most
// tiles then leave O where it is.
//
// Roundings: P to the inputs' type for the tensor cores, the result once; l sums the weights
// in fp32 before their rounding.  fp16 weights are scaled by 2^7, so that they keep full
// precision down to 2^-21 of the largest and stay below 2^15.
//
// Roles.  Two warpgroups for the softmax, one for each of two slots (S, P in its place, and O
// in TMEM); of the other warps one walks through the CTA's units and fetches their queries,
// one fetches tiles of keys and one of values (TMA; two each by 16-byte copies for pages that
// are no multiple of 8 slots: 4 x 1000 tokens over 2000 keys, 8 of 32 heads, d = 64, take 84 us
// with pages of 20 slots and 73 with 16; single tokens of 64 rows over 2000 keys, 4 of 16 heads,
// d = 128, 74 and 53), one issues all products, a slot's under the other's softmax.
//
// Bounds, and what the kernel comes to on the device.  Single tokens: the bytes of the cache,
// 32 rows over 8192 keys, 8 of 32 heads, 165 us at d = 128 (6.5 TB/s), 99 at d = 64 (5.4; up to
// 120 on a card that has just run long chunks), 74 at d = 32 (3.6).
// Long chunks at d = 128: the tensor cores, 4100 tokens over 32100 keys, 32 heads, 1.17 ms,
// 1.73 PFLOP/s.  At d = 64 the chain of a tile, S, maximum, exponentials, P, O, some 2400
// cycles for two slots' tiles where the tensor cores and the exponentials need 1050 each.
// Short calls: 4 to 5 us until the first tile has arrived and 4 to 6 for the join.  Two warps for
// the halves of a row (16 for the softmax), which swap their maxima, took a third longer at
// d = 128 and a tenth at d = 64.
#include <algorithm>
#include <cstring>
#include <numeric>

#include "gdn_attention.cuh"

namespace gdn {
namespace attn {
namespace {

using namespace tc;

constexpr int KT = 128;             // keys of a tile
constexpr int kThreads = 512;
// registers a thread: 128 at launch, of which two warpgroups give 72 each to the others
constexpr int kSoftmaxRegs = 200, kOtherRegs = 56;
constexpr uint32_t kBlock = 16384;  // 128 rows of 64 elements
constexpr uint32_t tS = 0, tO = 256;  // TMEM: S (and P in its place) and O of a slot, 128 columns each
constexpr uint32_t kTmemCols = 512;
constexpr float kGrowth = 8.f;      // of the maximum's exponent, before O follows
constexpr int kUnits = 4;           // units ahead

// Two ways to use the two slots (S and O in TMEM and a warpgroup each):
//  kPair   a unit has two blocks of up to 128 query rows, a slot each, which share the tiles
//  kOne    a unit has one block; the slots take its tiles in turn and are added up at the end
enum Mode { kPair, kOne };

// Shared memory: queries (blocks of 64 features, 128 rows each; kPair: both slots' of a unit,
// kOne: of two units in turn), the rings of tiles of keys and of values (8 keys x 64 features
// a kilobyte, all features of 8 keys together), and what the warps tell each other.
template <int NB>
struct Layout {
    static constexpr uint32_t kTile = NB * kBlock;
    static constexpr int NK = NB == 2 ? 3 : 5, NV = NB == 2 ? 2 : 5;  // tiles of keys, and of values, in flight
    static constexpr uint32_t oK = 2 * kTile, oV = oK + NK * kTile;
    static constexpr uint32_t oMerge = oV + NV * kTile;    // [128] maxima and sums of slot 1 (kOne)
    static constexpr uint32_t oWork = oMerge + 1024;       // [kUnits] Work
    static constexpr uint32_t oBar = oWork + kUnits * 96;
    // Barriers, each kind behind the one before; then the address that TMEM's allocation writes
    static constexpr int bKFull = 0, bKEmpty = bKFull + NK, bVFull = bKEmpty + NK, bVEmpty = bVFull + NV;
    static constexpr int bUFull = bVEmpty + NV, bUEmpty = bUFull + kUnits, bQFull = bUEmpty + kUnits;
    static constexpr int bQFree = bQFull + 2, bSFull = bQFree + 2, bPReady = bSFull + 2, bODone = bPReady + 2;
    static constexpr int bOther = bODone + 2, bMerged = bOther + 1, bDrain = bMerged + 1, kBars = bDrain + 1;
    static constexpr uint32_t oTmem = oBar + 8 * kBars;
    static constexpr uint32_t kSmem = oTmem + 16 + 1024;   // + alignment slack
    static_assert(kSmem <= 227 * 1024, "a CTA has no more shared memory");
};

struct TcParams : AttentionParams {
    explicit TcParams(const AttentionParams &p) : AttentionParams(p), page_size_((uint32_t)p.page_size) {}
    Plan plan;
    int slot_tokens;        // tokens of a slot
    int box;                // keys of a TMA box: the power of two in the page size
    Divisor page_size_;     // by the page's slots
    int box_log2;
    int page_step, head_step, none;  // a page's and a head's index in the maps, and one past all
    float c;                // |scale| log2 e
    uint32_t limit;         // of waits, ns: wait_ns, 4 s at most
};

// A piece's unit, as the warp that walks through them describes it.
struct Work {
    int n;             // tiles of the piece; 0: no keys; -1: no more units
    int key0;          // the first one's first key
    int lo, hi;        // keys that any query of the unit sees
    int b, hk, head0, heads;
    int a[2], e[2];    // tiles of each slot, from the piece's first one
    int tokens[2];     // tokens of each slot
    int pos, keys;     // cache position of the first token; keys of the row
    int part;          // of the CTA, that is left for the join; -1: none
    long tok0;         // the first token
};
static_assert(sizeof(Work) <= 96, "");

template <typename E>
struct Half16;
template <>
struct Half16<__nv_bfloat16> {
    static constexpr bool kBf16 = true;
    static constexpr float kShift = 0.f;
    __device__ static uint32_t pack2(float a, float b) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
};
template <>
struct Half16<__half> {
    static constexpr bool kBf16 = false;
    static constexpr float kShift = 7.f;
    __device__ static uint32_t pack2(float a, float b) {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t *>(&h);
    }
};

// Four lanes' four values, transposed: value r of lane t (of four in a row) to value t of lane r.
__device__ __forceinline__ void transpose4(uint32_t (&v)[4], int lane) {
#pragma unroll
    for (int b = 1; b <= 2; b <<= 1) {
        const bool up = (lane & b) != 0;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (r & b) continue;
            const uint32_t got = __shfl_xor_sync(kAll, up ? v[r] : v[r | b], b);
            if (up) v[r] = got;
            else v[r | b] = got;
        }
    }
}

// The unit at hand of a walk.
template <int MODE>
__device__ __forceinline__ Work work_of(const TcParams &p, const Walk<KT> &w) {
    Work x;
    const Unit &u = w.unit;
    x.n = u.hi > u.lo ? w.end - w.at.tile : 0;
    x.key0 = u.key0 + w.at.tile * KT;
    x.lo = u.lo;
    x.hi = u.hi;
    x.b = w.at.b;
    x.hk = w.key_head(p.plan);
    x.head0 = w.head0(p, p.plan);
    x.heads = w.heads(p, p.plan);
    x.pos = w.row.first + u.t0;
    x.keys = w.row.keys;
    x.part = w.part();
    x.tok0 = w.row.tok0 + u.t0;
#pragma unroll
    for (int s = 0; s < 2; ++s) {
        const int t = MODE == kPair ? s * p.slot_tokens : 0;
        x.tokens[s] = max(0, min(p.slot_tokens, u.t1 - u.t0 - t));
        int lo = u.lo, hi = u.hi;
        if (MODE == kPair && p.causal) {
            hi = min(hi, x.pos + t + x.tokens[s]);
            lo = max(lo, window_start(p, x.pos + t));
        }
        const bool any = x.n > 0 && x.tokens[s] > 0 && hi > lo;
        x.a[s] = any ? min(x.n, max(0, (lo - x.key0) >> 7)) : 0;
        x.e[s] = any ? max(x.a[s], min(x.n, (hi - x.key0 + KT - 1) >> 7)) : 0;
    }
    return x;
}

template <typename E, int NB, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const TcParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv) {
    using H = Half16<E>;
    using L = Layout<NB>;
    constexpr int NK = L::NK, NV = L::NV;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_align1k(smem_raw);
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::oBar);
    uint64_t *k_full = bars + L::bKFull, *k_empty = bars + L::bKEmpty, *v_full = bars + L::bVFull;
    uint64_t *v_empty = bars + L::bVEmpty, *u_full = bars + L::bUFull, *u_empty = bars + L::bUEmpty;
    uint64_t *q_full = bars + L::bQFull, *q_free = bars + L::bQFree;  // (kPair: the first of each)
    uint64_t *s_full = bars + L::bSFull, *p_ready = bars + L::bPReady, *o_done = bars + L::bODone;  // of a slot each
    uint64_t *other = bars + L::bOther, *merged = bars + L::bMerged, *drain = bars + L::bDrain;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(sm + L::oTmem);
    Work *works = reinterpret_cast<Work *>(sm + L::oWork);
    const bool gather = p.box < 8;  // pages that TMA boxes do not fit
    const int warp = __shfl_sync(kAll, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NK; ++i) {
            mbar_init(&k_full[i], gather ? 2 : 1);
            mbar_init(&k_empty[i], 1);
        }
        for (int i = 0; i < NV; ++i) {
            mbar_init(&v_full[i], gather ? 2 : 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < kUnits; ++i) {
            mbar_init(&u_full[i], 1);
            mbar_init(&u_empty[i], 8 + 3 + (gather ? 2 : 0));  // softmax, loading, issuing warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 1);
            mbar_init(&q_free[i], 1);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_ready[i], 4);
            mbar_init(&o_done[i], 1);
        }
        mbar_init(other, 4);
        mbar_init(merged, 4);
        mbar_init(drain, 1);
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, kTmemCols);
        tmem_relinquish();
    }
    grid_launch_dependents();
    const Place from = find_place<KT, kThreads>(p, p.plan);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = __shfl_sync(kAll, *tmem_slot, 0);
    bool ok = true;
    // Waits run out p.limit nanoseconds after the warp's last unit came (a tile takes about a
    // microsecond).  A wait of a whole warp, for a barrier's n-th completion (from 0): the same
    // outcome in every lane.
    uint32_t since = globaltimer_lo();
    auto wait = [&](uint64_t *bar, int n) {
        return __all_sync(kAll, mbar_wait_since(bar, (uint32_t)n & 1u, since, p.limit)) != 0;
    };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // The u-th unit; false past the last one.  (A limit below a microsecond, a test's, gives up
    // where it is not there yet, which the first one never is.)
    auto next_unit = [&](int u, Work &x) {
        ok = p.limit >= 1000 ? wait(&u_full[u % kUnits], u / kUnits)
                             : __all_sync(kAll, mbar_test_wait(&u_full[u % kUnits], (uint32_t)(u / kUnits) & 1u)) != 0;
        if (!ok) return false;
        since = globaltimer_lo();
        x = works[u % kUnits];
        arrive(&u_empty[u % kUnits]);
        return x.n >= 0;
    };

    if (warp < 8) {
        // ============================ softmax ============================
        regs_inc<kSoftmaxRegs>();
        const int s = warp >> 2, r = (warp & 3) * 32 + lane;  // slot, row of the slot
        const int t = r / p.plan.gs, g = r - t * p.plan.gs;   // its token in the slot, its head in the group
        const uint32_t lanes = tm + ((uint32_t)((warp & 3) * 32) << 16);
        const uint32_t ts = lanes + tS + 128 * s, to = lanes + tO + 128 * s;
        float2 *merge = reinterpret_cast<float2 *>(sm + L::oMerge);
        const float2 c2 = make_float2(p.c, p.c);
        const int slot_t = MODE == kPair ? s * p.slot_tokens : 0;
        const int row = slot_t * p.plan.gs + r;  // of the unit
        int item = 0, merges = 0;
        Work x;
#pragma unroll 1
        for (int u = 0; next_unit(u, x); ++u) {
            const int tokens = s ? x.tokens[1] : x.tokens[0];
            const bool mine = t < tokens && g < x.heads;
            const bool idle = (warp & 3) * 32 >= tokens * p.plan.gs;  // the whole warp has no row
            int lo = 0, hi = 0x7fffffff;  // keys that the row sees (rows that are not there: any)
            if (mine) {
                hi = x.keys;
                if (p.causal) {
                    const int at = x.pos + slot_t + t;
                    hi = min(hi, at + 1);
                    lo = window_start(p, at);
                }
            }
            float m = kNone, l = 0.f;  // m: c times the score that weights are relative to
            const int i0 = MODE == kOne ? s : s ? x.a[1] : x.a[0], i1 = MODE == kOne ? x.n : s ? x.e[1] : x.e[0];
#pragma unroll 1
            for (int i = i0; i < i1; i += MODE == kPair ? 1 : 2, ++item) {
                if (!(ok = wait(&s_full[s], item))) break;
                fence_after_sync();
                if (idle) {
                    arrive(&p_ready[s]);
                    continue;
                }
                uint32_t v[4][32];
#pragma unroll
                for (int j = 0; j < 4; ++j) tmem_ld32_async(ts + 32 * j, v[j]);
                tmem_wait_ld();
                const int a = lo - (x.key0 + i * KT), e = hi - (x.key0 + i * KT);
                if (__any_sync(kAll, e < KT)) {
#pragma unroll
                    for (int j = 0; j < KT; ++j)
                        if (j >= e) v[j >> 5][j & 31] = 0xff800000u;
                }
                if (__any_sync(kAll, a > 0)) {
#pragma unroll
                    for (int j = 0; j < KT; ++j)
                        if (j < a) v[j >> 5][j & 31] = 0xff800000u;
                }
                float top[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) top[j] = __uint_as_float(v[j][0]);
#pragma unroll
                for (int k = 1; k < 32; ++k)
#pragma unroll
                    for (int j = 0; j < 4; ++j) top[j] = fmaxf(top[j], __uint_as_float(v[j][k]));
                const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.c;
                const bool grow = now - m > kGrowth;  // (from none: always, unless there is still none)
                if (__any_sync(kAll, grow)) {
                    const float keep = grow ? ex2_approx(m - now) : 1.f;
                    m = grow ? now : m;
                    if (i != i0) {
                        // (the slot's last product is done: S was issued behind it)
                        l *= keep;
                        const float2 k2 = make_float2(keep, keep);
#pragma unroll 1
                        for (int j = 0; j < p.d; j += 16) {
                            uint32_t o[16];
                            tmem_ld16_async(to + j, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; k += 2) {
                                const float2 y = __fmul2_rn(k2, make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])));
                                o[k] = __float_as_uint(y.x);
                                o[k + 1] = __float_as_uint(y.y);
                            }
                            tmem_st16(to + j, o);
                        }
                    }
                }
                // (held finite: without keys so far weights are 0)
                const float off = H::kShift - fmaxf(m, -3.4028235e38f);
                const float2 off2 = make_float2(off, off);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t pk[16];
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        float2 y = __ffma2_rn(make_float2(__uint_as_float(v[j][k]), __uint_as_float(v[j][k + 1])), c2, off2);
                        y.x = ex2_approx(y.x);
                        y.y = ex2_approx(y.y);
                        sum[(k >> 1) & 1] = __fadd2_rn(sum[(k >> 1) & 1], y);
                        pk[k / 2] = H::pack2(y.x, y.y);
                    }
                    tmem_st16(ts + 16 * j, pk);
                }
                tmem_wait_st();
                fence_before_sync();
                arrive(&p_ready[s]);
                sum[0] = __fadd2_rn(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
            }
            if (!ok) break;
            const bool any = i1 > i0;  // the slot has sums of its own
            if (any) {
                if (!(ok = wait(&o_done[s], item - 1))) break;
                fence_after_sync();
            }
            float f0 = 1.f, f1 = 0.f;  // factors of this slot's sums, and of the other's (kOne)
            const bool both = MODE == kOne && x.n > 1;
            if (both) {
                if (s == 1) {
                    merge[r] = make_float2(m, l);
                    arrive(other);
                    // (the next unit's products here wait for what the others read)
                    if (!(ok = wait(merged, merges++))) break;
                    continue;
                }
                if (!(ok = wait(other, merges++))) break;
                fence_after_sync();
                const float2 ml = merge[r];
                const float top = fmaxf(m, ml.x), safe = top == kNone ? 0.f : top;
                f0 = ex2_approx(m - safe);
                f1 = ex2_approx(ml.x - safe);
                m = top;
                l = f0 * l + f1 * ml.y;
            } else if (MODE == kOne && s == 1) {
                continue;
            }
            if (!idle) {
                const bool whole = x.part < 0;
                const float inv = !whole ? 1.f : l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // (a NaN stays one)
                f0 *= inv;
                f1 *= inv;
                const long at = (x.tok0 + slot_t + t) * p.Hq + x.head0 + g;
                if (mine) {
                    if (!whole) p.plan.stats(blockIdx.x, x.part)[row] = make_float2(m - H::kShift, l);
                    else if (p.lse != nullptr)
                        p.lse[at] = ((m == kNone ? 0.f : m - H::kShift) + log2f(l)) * 0.69314718055994530942f;
                }
                // O leaves TMEM as fragments, lane 4 g + t: columns 2 t, 2 t + 1 of every 8 of rows
                // g and g + 8, and is transposed between four lanes, which then write 8 columns
                // each: 8 rows a store.  (A row a lane, stores of 32 rows took 2 us a unit, parts
                // in fp32 5 us.)
                const unsigned there = __ballot_sync(kAll, mine);
                char *to_row = whole ? static_cast<char *>(p.out) + at * p.d * (long)sizeof(E)
                                     : reinterpret_cast<char *>(p.plan.sums(blockIdx.x, x.part & 1) + row * p.d);
#pragma unroll 1
                for (int turn = 0; turn < 2 * NB; ++turn) {  // 16 rows, 64 columns
                    const int c = turn / NB, col = turn % NB * 64;
                    if ((there >> (16 * c) & 0xffff) == 0) continue;
                    const uint32_t from = to + ((uint32_t)(16 * c) << 16) + col;
                    float2 y[2][2][4];  // of rows g and g + 8: 32 columns a time, 8 r + 2 t
                    __syncwarp();
#pragma unroll
                    for (int part = 0; part < (MODE == kOne ? 2 : 1); ++part) {
                        if (part == 1 && !both) break;
                        uint32_t o[2][16];
#pragma unroll
                        for (int q = 0; q < 2; ++q)
                            if (32 * q < p.d) tmem_ld_16x32(from + part * 128 + 32 * q, o[q]);
                        tmem_wait_ld();
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float f = __shfl_sync(kAll, part ? f1 : f0, 16 * c + 8 * h + (lane >> 2));
#pragma unroll
                            for (int q = 0; q < 2; ++q)
#pragma unroll
                                for (int r = 0; r < 4; ++r) {
                                    const float2 v = make_float2(__uint_as_float(o[q][4 * r + 2 * h]),
                                                                 __uint_as_float(o[q][4 * r + 2 * h + 1]));
                                    // (without sums of its own the slot's columns hold anything)
                                    if (part == 0) y[h][q][r] = any ? __fmul2_rn(v, make_float2(f, f)) : make_float2(0.f, 0.f);
                                    else y[h][q][r] = __ffma2_rn(v, make_float2(f, f), y[h][q][r]);
                                }
                        }
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int of = 16 * c + 8 * h + (lane >> 2);
                        char *dst = reinterpret_cast<char *>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(to_row), of)) +
                                    (col + 8 * (lane & 3)) * (whole ? sizeof(E) : sizeof(float));
                        const bool write = there >> of & 1;
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            if (32 * q >= p.d) break;
                            if (whole) {
                                uint32_t v[4];
#pragma unroll
                                for (int r = 0; r < 4; ++r) v[r] = H::pack2(y[h][q][r].x, y[h][q][r].y);
                                transpose4(v, lane);
                                if (write) *reinterpret_cast<uint4 *>(dst + 64 * q) = make_uint4(v[0], v[1], v[2], v[3]);
                            } else {
                                uint32_t a[4], b[4];
#pragma unroll
                                for (int r = 0; r < 4; ++r)
                                    a[r] = __float_as_uint(y[h][q][r].x), b[r] = __float_as_uint(y[h][q][r].y);
                                transpose4(a, lane);
                                transpose4(b, lane);
                                if (write) {
                                    *reinterpret_cast<uint4 *>(dst + 128 * q) = make_uint4(a[0], b[0], a[1], b[1]);
                                    *reinterpret_cast<uint4 *>(dst + 128 * q + 16) = make_uint4(a[2], b[2], a[3], b[3]);
                                }
                            }
                        }
                    }
                }
                fence_before_sync();
            }
            if (both) arrive(merged);
        }
        tmem_wait_st();  // (given up or not, TMEM is freed behind the stores)
    } else {
        regs_dec<kOtherRegs>();
        const uint32_t leader = elect_leader();
        if (gather && (warp & 1) == 0) {
            // ====== loads, keys or values: pages of any size, 16 bytes a lane ======
            // Two warps a tile, 64 rows each.  The copies are this thread's own writes: it waits
            // for them and passes them to the tensor cores' side with a fence, a tile behind.
            constexpr int kCols = 8 * NB;  // 16-byte columns of a row (of 32 elements: 4)
            const bool values = (warp & 2) != 0;
            const int r0 = warp >= 12 ? 64 : 0;
            uint64_t *full = values ? v_full : k_full, *empty = values ? v_empty : k_empty;
            const char *pages = static_cast<const char *>(values ? p.v_pages : p.k_pages);
            uint8_t *ring = sm + (values ? L::oV : L::oK);
            const int stages = values ? NV : NK;
            int st = 0, round = 0, pending = -1;  // of the ring; the stage that is not handed on yet
            auto hand_on = [&]() {
                if (pending < 0) return;
                fence_proxy_async();
                arrive(&full[pending]);
                pending = -1;
            };
            auto landed = [&]() {
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                hand_on();
            };
            Work x;
#pragma unroll 1
            for (int u = 0; next_unit(u, x); ++u) {
                const int32_t *table = p.page_table + (int64_t)x.b * p.max_pages;
                // Pages of the lane's rows (lane, lane + 32 of the warp's), read a tile ahead
                auto page_of = [&](int i, int h) {
                    const int k = x.key0 + i * KT + r0 + 32 * h + lane;
                    return i < x.n && k >= x.lo && k < x.hi ? table[p.page_size_.div((uint32_t)k)] : -1;
                };
                int ahead[2] = {page_of(0, 0), page_of(0, 1)};
#pragma unroll 1
                for (int i = 0; i < x.n; ++i) {
                    const int k0 = x.key0 + i * KT + r0;
                    long row[2];  // bytes into the pages; -1: left out, -2: zeros
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int k = k0 + 32 * h + lane, page = ahead[h];
                        row[h] = -1;
                        if (k >= x.lo && k < x.hi) {
                            row[h] = -2;
                            if (page >= 0 && page < p.num_pages)
                                row[h] = 2 * (page * p.page_stride + (long)p.page_size_.rest((uint32_t)k) * p.slot_stride +
                                              x.hk * p.head_stride);
                            else atomicOr(p.err, (uint32_t)GDN_DEVERR_BAD_INDEX);
                        }
                        ahead[h] = page_of(i + 1, h);
                    }
                    if (round > 0) {
                        // (all lanes or none: it holds the warp's barrier and its one arrival)
                        if (__any_sync(kAll, !mbar_test_wait(&empty[st], (uint32_t)(round - 1) & 1u))) landed();
                        if (!(ok = wait(&empty[st], round - 1))) break;
                    }
                    uint8_t *dst = ring + st * L::kTile + (r0 >> 3) * (NB * 1024);
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll 4
                        for (int y = 0; y < kCols; ++y) {
                            const int at = y * 32 + lane, r = at / kCols, c = at % kCols;  // row of 32, column
                            const long from = __shfl_sync(kAll, row[h], r);
                            if (from == -1 || 8 * c >= p.d) continue;
                            const int q = 32 * h + r;
                            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                             smem_u32(dst + (q >> 3) * (NB * 1024) + (c >> 3) * 1024 + sw128_chunk(q & 7, c & 7))),
                                         "l"(pages + (from < 0 ? 0 : from + 16 * c)), "r"(from < 0 ? 0 : 16)
                                         : "memory");
                        }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    if (pending >= 0) {
                        asm volatile("cp.async.wait_group 1;" ::: "memory");
                        hand_on();
                    }
                    pending = st;
                    if (++st == stages) st = 0, ++round;
                }
                if (!ok) break;
                landed();
            }
            landed();
        } else if (warp == 8 || warp == 10) {
            // ================== loads: keys, or values ===================
            const bool values = warp == 10;
            const int boxes = KT / p.box;  // (pages of a multiple of 8 slots)
            // This lane's box of a tile.  Its page is read a tile ahead.
            const int first = lane * p.box;
            uint64_t *full = values ? v_full : k_full, *empty = values ? v_empty : k_empty;
            uint8_t *ring = sm + (values ? L::oV : L::oK);
            const int stages = values ? NV : NK;
            int st = 0, round = 0;  // of the ring
            Work x;
#pragma unroll 1
            for (int u = 0; next_unit(u, x); ++u) {
                const int32_t *table = p.page_table + (int64_t)x.b * p.max_pages;
                auto page_of = [&](int i) {
                    const int k = x.key0 + i * KT + first;
                    return i < x.n && lane < boxes && k + p.box > x.lo && k < x.hi ? table[p.page_size_.div((uint32_t)k)]
                                                                                   : -1;
                };
                int ahead = page_of(0);
#pragma unroll 1
                for (int i = 0; i < x.n; ++i) {
                    const int k0 = x.key0 + i * KT, k = k0 + first;
                    const int b0 = (max(x.lo, k0) - k0) >> p.box_log2, b1 = (min(x.hi - k0, KT) + p.box - 1) >> p.box_log2;
                    int index = p.none;  // of this lane's box (one past all: zeros)
                    if (lane >= b0 && lane < b1) {
                        if (ahead >= 0 && ahead < p.num_pages) index = ahead * p.page_step + x.hk * p.head_step;
                        else atomicOr(p.err, (uint32_t)GDN_DEVERR_BAD_INDEX);
                    }
                    const int slot = (int)p.page_size_.rest((uint32_t)k) >> 3;
                    ahead = page_of(i + 1);
                    if (round > 0 && !(ok = wait(&empty[st], round - 1))) break;
                    if (leader) mbar_arrive_expect_tx(&full[st], (uint32_t)((b1 - b0) * p.box * 128 * NB));
                    __syncwarp();
                    uint8_t *dst = ring + st * L::kTile;
                    // (by the converged warp, a box after the other: lanes that issue their own
                    // box each take 60 ns for it)
#pragma unroll 2
                    for (int y = b0; y < b1; ++y)
                        tma_load_5d_warp(leader, dst + y * p.box * (128 * NB), values ? &mv : &mk, 0, 0, 0,
                                         __shfl_sync(kAll, slot, y), __shfl_sync(kAll, index, y), &full[st]);
                    __syncwarp();
                    if (++st == stages) st = 0, ++round;
                }
                if (!ok) break;
            }
            // The copies in flight land before the CTA ends, whoever gave up.
            __syncwarp();
#pragma unroll 1
            for (int y = 0; y < stages; ++y) {
                const int n = y < st ? round : round - 1;  // the stage's last load
                if (n >= 0) mbar_wait(&full[y], (uint32_t)n & 1u, kDefaultWaitNs / 8);
            }
        } else if (warp == 11) {
            // =================== units, and their queries ================
            Walk<KT> w;
            Cut cut{};
            bool more = w.start(p, p.plan, from);
            int live = 0;  // units with keys
            const uint32_t bytes = (uint32_t)(p.slot_tokens * p.plan.gs) * 128 * NB * (MODE == kPair ? 2 : 1);
#pragma unroll 1
            for (int u = 0;; ++u) {
                if (u >= kUnits && !(ok = wait(&u_empty[u % kUnits], u / kUnits - 1))) break;
                since = globaltimer_lo();
                Work x;
                x.n = -1;
                if (more) x = work_of<MODE>(p, w);
                if (lane == 0) works[u % kUnits] = x;
                arrive(&u_full[u % kUnits]);
                if (!more) break;
                if (x.n > 0) {
                    const int buf = MODE == kOne ? live & 1 : 0, turn = MODE == kOne ? live >> 1 : live;
                    if (turn > 0 && !(ok = wait(&q_free[buf], turn - 1))) break;
                    since = globaltimer_lo();
                    if (leader) {
                        mbar_arrive_expect_tx(&q_full[buf], bytes);
#pragma unroll 1
                        for (int y = 0; y < (MODE == kPair ? 2 * NB : NB); ++y)
                            tma_load_3d(sm + buf * L::kTile + y * kBlock, &mq, 64 * (y % NB), x.head0,
                                        (int)x.tok0 + y / NB * p.slot_tokens, &q_full[buf]);
                    }
                    __syncwarp();
                    ++live;
                }
                cut = w.cut(p, p.plan);
                more = w.next(p, p.plan);
            }
            if (lane == 0) *p.plan.cut(blockIdx.x) = cut;
            // (a barrier's last completion: older ones are not told from none)
            for (int x = max(0, live - (MODE == kOne ? 2 : 1)); x < live; ++x)
                mbar_wait(&q_full[MODE == kOne ? x & 1 : 0], (uint32_t)(MODE == kOne ? x >> 1 : x) & 1u, kDefaultWaitNs / 8);
        } else if (warp == 9) {
            // ============================ MMAs ===========================
            // One warp issues all, slot after slot, so that one slot's softmax runs under the
            // other's products (a warp a slot: both ran in step, 1403 us where one takes 1183).
            // (a negative scale: of the scores' queries)
            const uint32_t id_s = idesc_f16(128, KT, false, false, H::kBf16) | (p.scale < 0.f ? 1u << 13 : 0u);
            const uint32_t id_o = idesc_f16(128, p.d, false, true, H::kBf16);
            const uint64_t q0 = desc_sw128(smem_u32(sm), 16, 1024);
            const uint64_t k0 = desc_sw128(smem_u32(sm) + L::oK, 16, NB * 1024);
            const uint64_t v0 = desc_sw128(smem_u32(sm) + L::oV, 1024, NB * 1024);
            int live = 0, items[2] = {0, 0};               // of a slot: sums so far
            int kst = 0, kround = 0, vst = 0, vround = 0;  // of the rings
            Work x;
#pragma unroll 1
            for (int u = 0; next_unit(u, x); ++u) {
                if (x.n == 0) continue;
                const int n = x.n, buf = MODE == kOne ? live & 1 : 0;
                if (!(ok = wait(&q_full[buf], MODE == kOne ? live >> 1 : live))) break;
                auto has = [&](int s, int i) {
                    return MODE == kOne ? i >= 0 && i < n && (i & 1) == s
                                        : i >= (s ? x.a[1] : x.a[0]) && i < (s ? x.e[1] : x.e[0]);
                };
                auto next = [&](int &st, int &round, int stages) {
                    if (++st == stages) st = 0, ++round;
                };
                // S of slot s = Q K_i^T, of the tile of keys at hand; `first`, `last`: of its uses
                auto scores = [&](int s, bool first, bool last) {
                    if (first && !(ok = wait(&k_full[kst], kround))) return;
                    fence_after_sync();
                    const uint64_t qd = desc_add(q0, (MODE == kOne ? buf : s) * L::kTile), kd = desc_add(k0, kst * L::kTile);
#pragma unroll
                    for (int k = 0; k < 4 * NB; ++k)
                        if (16 * k < p.d)
                            mma_f16_warp(leader, tm + tS + 128 * s, desc_add(qd, (k >> 2) * kBlock + (k & 3) * 32),
                                         desc_add(kd, (k >> 2) * 1024 + (k & 3) * 32), id_s, k > 0);
                    mma_commit_warp(leader, &s_full[s]);
                    if (last) {
                        mma_commit_warp(leader, &k_empty[kst]);
                        next(kst, kround, NK);
                    }
                };
                // O of slot s += P V_i, of the tile of values at hand
                auto sums = [&](int s, int i, bool first, bool last) {
                    if (first) {
                        if (!(ok = wait(&v_full[vst], vround))) return;
                        // Values of keys that no query of the unit sees: zeros, whatever was
                        // there (their weights are 0, but 0 times NaN is not).
                        const int key = x.key0 + i * KT;
                        const int r0 = max(0, x.lo - key), r1 = min(KT, x.hi - key);
                        if (r0 > 0 || r1 < KT) {
                            uint8_t *v = sm + L::oV + vst * L::kTile;
#pragma unroll 1
                            for (int y = lane; y < (r0 + KT - r1) * 8 * NB; y += 32) {
                                int row = y / (8 * NB);
                                row = row < r0 ? row : row - r0 + r1;
                                *reinterpret_cast<uint4 *>(v + (row >> 3) * (NB * 1024) + (y / 8 % NB) * 1024 +
                                                           (row & 7) * 128 + (y & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                            }
                            fence_proxy_async();
                            __syncwarp();
                        }
                    }
                    if (!(ok = wait(&p_ready[s], s ? items[1] : items[0]))) return;
                    if (s) ++items[1];
                    else ++items[0];
                    fence_after_sync();
                    const uint64_t vd = desc_add(v0, vst * L::kTile);
                    const uint32_t more = has(s, i - (MODE == kPair ? 1 : 2));
#pragma unroll
                    for (int k = 0; k < KT / 16; ++k)
                        mma_f16_ta_warp(leader, tm + tO + 128 * s, tm + tS + 128 * s + 8 * k,
                                        desc_add(vd, k * NB * 2048), id_o, k > 0 ? 1u : more);
                    mma_commit_warp(leader, &o_done[s]);
                    if (last) {
                        mma_commit_warp(leader, &v_empty[vst]);
                        next(vst, vround, NV);
                    }
                };
                // Turn y, for slot s = y % 2: sums of tile i, and scores of the slot's next tile.
                // (kOne: i = y - 2, the tiles in turn; kPair: both slots have tile i = y / 2 - 1.)
#pragma unroll 1
                for (int y = 0; ok && y < (MODE == kOne ? n + 2 : 2 * n + 2); ++y) {
                    const int s = y & 1, i = MODE == kOne ? y - 2 : (y >> 1) - 1, to_come = MODE == kOne ? y : i + 1;
                    const bool both_sums = MODE == kPair && has(0, i) && has(1, i);
                    const bool both_scores = MODE == kPair && has(0, to_come) && has(1, to_come);
                    if (has(s, i)) sums(s, i, !both_sums || s == 0, !both_sums || s == 1);
                    if (ok && has(s, to_come)) scores(s, !both_scores || s == 0, !both_scores || s == 1);
                    // the unit's last scores are issued
                    if (ok && y == (MODE == kOne ? n : 2 * n) - 1) mma_commit_warp(leader, &q_free[buf]);
                }
                if (!ok) break;
                ++live;
            }
            mma_commit_warp(leader, drain);  // nothing may be in flight when TMEM is given back
            mbar_wait(drain, 0, kDefaultWaitNs);
        }
    }
    if (!ok && lane == 0) atomicOr(p.err, (uint32_t)GDN_DEVERR_TIMEOUT);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    if (warp == 0) tmem_dealloc(tm, kTmemCols);
}

template <typename E, int NB, int MODE>
cudaError_t launch_mode(const TcParams &p, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                        cudaStream_t stream) {
    constexpr uint32_t bytes = Layout<NB>::kSmem;
    cudaError_t e = set_smem_once<attention_kernel<E, NB, MODE>>((int)bytes);
    if (e != cudaSuccess) return e;
    attention_kernel<E, NB, MODE><<<p.plan.ctas, kThreads, bytes, stream>>>(p, mq, mk, mv);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join(p, p.plan, stream);
}

template <typename E, int NB>
cudaError_t launch_nb(const TcParams &p, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                      cudaStream_t stream) {
    return p.plan.tokens > p.slot_tokens ? launch_mode<E, NB, kPair>(p, mq, mk, mv, stream)
                                         : launch_mode<E, NB, kOne>(p, mq, mk, mv, stream);
}

// A page's and a head's steps in the one dimension that the maps have for both, in units of
// their strides' common divisor (a dimension of one has no stride).
struct Steps {
    int64_t unit, page, head, count;
};
Steps steps_of(const AttentionParams &p) {
    const int64_t ps = p.num_pages > 1 ? p.page_stride : 0, hs = p.Hk > 1 ? p.head_stride : 0;
    Steps x{};
    x.unit = std::gcd(ps, hs);
    if (x.unit == 0) x.unit = p.d;
    x.page = ps / x.unit;
    x.head = hs / x.unit;
    const int64_t limit = 1ll << 31;
    if (x.page < limit && x.head < limit) x.count = (p.num_pages - 1) * x.page + (p.Hk - 1) * x.head + 1;
    else x.count = limit;
    return x;
}

}  // namespace

bool tc_takes(const AttentionParams &p) {
    if (p.dt == GDN_F32 || p.num_pages == 0) return false;
    // tensor maps, and 16-byte copies: addresses and strides of 16 bytes, strides below 2^40 bytes, indexes of 31 bits
    const uint64_t all = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k_pages) |
                         reinterpret_cast<uintptr_t>(p.v_pages) |
                         (uint64_t)(p.qs | p.page_stride | p.slot_stride | p.head_stride) * 2;
    if ((all & 15) != 0) return false;
    const int64_t limit = 1ll << 36;  // (a slot's stride is taken times 8)
    return p.qs < limit && p.page_stride < limit && p.slot_stride < limit && p.head_stride < limit &&
           steps_of(p).count < (1ll << 31) - 1;
}

// One block a unit, or two that share its tiles: two where there are as many blocks as CTAs.
// With fewer every unit is cut, and pairs have twice the rows to leave and to join; with more,
// tiles are fetched half as often and the slots' sums need no adding up.  us with one and with
// two a unit, 4 of 16 heads, tokens of a row after 2000 others:
//     d = 64:  1 x 512 (64 blocks)  22, 26;   8 x 128 (128)  26, 28;   64 x 512 (4096)  371, 328
//     d = 128: 1 x 512              27, 29;   8 x 128        34, 32;   64 x 512         774, 456
Plan plan_tc(int B, int T, int Hq, int Hk, int d, bool varlen) {
    const int ctas = sm_count_of_current_device();
    Plan s = plan_of(Hq, Hk, d, 128, ctas, 2, 1);
    const long mean = mean_tokens(B, T, varlen), blocks = (mean + s.tokens - 1) / s.tokens;
    if (blocks > 1 && blocks * B * Hk * s.per_key >= ctas) s.tokens *= 2;
    return s;
}

cudaError_t launch_attention_tc(const AttentionParams &pp, const Plan &plan, cudaStream_t stream) {
    TcParams p(pp);
    p.plan = plan;
    p.slot_tokens = 128 / plan.gs;
    p.box = std::min(KT, p.page_size & -p.page_size);
    p.box_log2 = 0;
    while (1 << p.box_log2 < p.box) ++p.box_log2;
    const Steps x = steps_of(pp);
    p.page_step = (int)x.page;
    p.head_step = (int)x.head;
    p.none = (int)x.count;
    // (a scale of 0 gives every key that is seen the same weight, and -infinity still none)
    p.c = std::max(std::abs(p.scale) * kLog2e, 0x1p-126f);
    p.limit = (uint32_t)std::min<uint64_t>(p.wait_ns, 4000000000ull);
    const long total = p.cu_seqlens != nullptr ? (long)p.T : (long)p.B * p.T;
    const bool bf = p.dt == GDN_BF16;
    CUtensorMap mq, mk, mv;
    memset(&mk, 0, sizeof(mk));
    memset(&mv, 0, sizeof(mv));
    if (!encode_heads_map(&mq, p.q, bf, p.d, p.Hq, total, p.qs, plan.gs, p.slot_tokens)) return cudaErrorInvalidValue;
    if (p.box >= 8 &&
        (!encode_pages_map(&mk, p.k_pages, bf, p.d, p.page_size, p.slot_stride, x.count, x.unit, p.box) ||
         !encode_pages_map(&mv, p.v_pages, bf, p.d, p.page_size, p.slot_stride, x.count, x.unit, p.box)))
        return cudaErrorInvalidValue;
    if (p.d == 128)
        return bf ? launch_nb<__nv_bfloat16, 2>(p, mq, mk, mv, stream) : launch_nb<__half, 2>(p, mq, mk, mv, stream);
    return bf ? launch_nb<__nv_bfloat16, 1>(p, mq, mk, mv, stream) : launch_nb<__half, 1>(p, mq, mk, mv, stream);
}

}  // namespace attn
}  // namespace gdn
