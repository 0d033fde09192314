// gdn_attention_tc.cu -- attention over a paged cache on the 5th-generation tensor cores
// (tcgen05 MMA, TMEM, TMA), for 16-bit tensors.
//
// Per query row, over tiles of 128 keys (x: raw scores, c = scale log2 e):
//     S = Q K^T,  m' = max(m, max_j S_j),  P_j = 2^{c S_j - c m'}
//     l <- 2^{c (m - m')} l + sum_j P_j,   O <- 2^{c (m - m')} O + P V
// and O / l at the end.  S and O are fp32 in TMEM, a query row to a lane, so a thread has a
// whole row of a tile: no reduction crosses threads.  m follows the true maximum only when
// that has grown by more than 8 in the exponent: weights of up to 2^8 are as exact, and most
// tiles then leave O where it is.
//
// Roundings: P to the inputs' type for the tensor cores, the result once; l sums the weights
// in fp32 before their rounding.  fp16 weights are scaled by 2^7, so that they keep full
// precision down to 2^-21 of the largest and stay below 2^15.
#include <algorithm>
#include <cstring>
#include <numeric>

#include "gdn_attention.cuh"

namespace gdn {
namespace attn {
namespace {

using namespace tc;

constexpr int KT = 128;             // keys of a tile
constexpr int kThreads = 384;
// registers a thread: 168 at launch, of which the third warpgroup gives 96 to the others
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
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
// kOne: of two units in turn), the ring of tiles (8 keys x 64 features a kilobyte; a row of 8
// keys has all its features together), and what the warps tell each other.
template <int NB>
struct Layout {
    static constexpr uint32_t kTile = NB * kBlock;
    static constexpr int NS = NB == 2 ? 5 : 10;            // tiles of keys or values in flight
    static constexpr uint32_t oKv = 2 * kTile;
    static constexpr uint32_t oMerge = oKv + NS * kTile;   // [128] maxima and sums of slot 1 (kOne)
    static constexpr uint32_t oWork = oMerge + 1024;       // [kUnits] Work
    static constexpr uint32_t oBar = oWork + kUnits * 96;
    static constexpr uint32_t kSmem = oBar + 384 + 1024;   // + alignment slack
};

struct TcParams : AttentionParams {
    Plan plan;
    int slot_tokens;        // tokens of a slot
    int box;                // keys of a TMA box: the power of two in the page size
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

// Order in which a piece's n tiles of keys and values go through the ring: the issuing warp's
// order of use.  kPair: K0 V0 K1 V1 ..; kOne, one tile of scores ahead: K0 K1 V0 K2 V1 K3 ..
template <int MODE>
__device__ __forceinline__ int seq_k(int i) { return MODE == kPair ? 2 * i : i == 0 ? 0 : 2 * i - 1; }
template <int MODE>
__device__ __forceinline__ int seq_v(int i, int n) { return MODE == kPair || i == n - 1 ? 2 * i + 1 : 2 * i + 2; }

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
            if (p.window > 0) lo = max(lo, x.pos + t - p.window + 1);
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
    constexpr int NS = L::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_align1k(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::oBar), *empty = full + NS;
    uint64_t *u_full = empty + NS, *u_empty = u_full + kUnits;
    uint64_t *q_full = u_empty + kUnits, *q_free = q_full + 2;  // (kPair: the first of each)
    uint64_t *s_full = q_free + 2, *p_ready = s_full + 2, *o_done = p_ready + 2;  // of a slot each
    uint64_t *other = o_done + 2, *merged = other + 1, *drain = other + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(other + 3);
    Work *works = reinterpret_cast<Work *>(sm + L::oWork);
    const int warp = __shfl_sync(kAll, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kUnits; ++i) {
            mbar_init(&u_full[i], 1);
            mbar_init(&u_empty[i], 8 + 3);  // softmax warps, two that load, one that issues MMAs
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
    // Waits run out p.limit nanoseconds after the warp's last unit or tile came.  A wait of a
    // whole warp, for a barrier's n-th completion (from 0): the same outcome in every lane.
    uint32_t since = globaltimer_lo();
    auto wait = [&](uint64_t *bar, int n) {
        return __all_sync(kAll, mbar_wait_since(bar, (uint32_t)n & 1u, since, p.limit)) != 0;
    };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    // The u-th unit; false past the last one.
    auto next_unit = [&](int u, Work &x) {
        if (!(ok = wait(&u_full[u % kUnits], u / kUnits))) return false;
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
        const uint32_t ts = tm + ((uint32_t)((warp & 3) * 32) << 16) + tS + 128 * s;
        const uint32_t to = tm + ((uint32_t)((warp & 3) * 32) << 16) + tO + 128 * s;
        float2 *merge = reinterpret_cast<float2 *>(sm + L::oMerge);
        const float2 c2 = make_float2(p.c, p.c);
        const int slot_t = MODE == kPair ? s * p.slot_tokens : 0;
        const int row = slot_t * p.plan.gs + r;  // of the unit
        int item = 0, done = 0, merges = 0;
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
                    if (p.window > 0) lo = max(0, at - p.window + 1);
                }
            }
            float m = kNone, l = 0.f;  // m: c times the score that weights are relative to
            const int i0 = MODE == kOne ? s : s ? x.a[1] : x.a[0], i1 = MODE == kOne ? x.n : s ? x.e[1] : x.e[0];
#pragma unroll 1
            for (int i = i0; i < i1; i += MODE == kPair ? 1 : 2, ++item) {
                if (!(ok = wait(&s_full[s], item))) break;
                since = globaltimer_lo();
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
                        // the slot's last product is done: S was issued behind it
                        l *= keep;
                        const float2 k2 = make_float2(keep, keep);
#pragma unroll
                        for (int j = 0; j < 4 * NB; ++j) {
                            if (16 * j < p.d) {
                                uint32_t o[16];
                                tmem_ld16_async(to + 16 * j, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int k = 0; k < 16; k += 2) {
                                    const float2 y =
                                        __fmul2_rn(k2, make_float2(__uint_as_float(o[k]), __uint_as_float(o[k + 1])));
                                    o[k] = __float_as_uint(y.x);
                                    o[k + 1] = __float_as_uint(y.y);
                                }
                                tmem_st16(to + 16 * j, o);
                            }
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
                if (!(ok = wait(&o_done[s], done))) break;
                ++done;
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
                E *out = reinterpret_cast<E *>(p.out) + at * p.d;
                float *left = p.plan.sums(blockIdx.x, x.part & 1) + row * p.d;
#pragma unroll 1
                for (int j = 0; j < p.d; j += 16) {
                    uint32_t o[16], o1[16];
                    float y[16];
                    if (any) tmem_ld16_async(to + j, o);
                    if (both) tmem_ld16_async(to + 128 + j, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        y[k] = any ? __uint_as_float(o[k]) * f0 : 0.f;
                        if (both) y[k] = fmaf(__uint_as_float(o1[k]), f1, y[k]);
                    }
                    if (mine && whole) {
#pragma unroll
                        for (int k = 0; k < 16; k += 8)
                            *reinterpret_cast<uint4 *>(out + j + k) =
                                make_uint4(H::pack2(y[k], y[k + 1]), H::pack2(y[k + 2], y[k + 3]),
                                           H::pack2(y[k + 4], y[k + 5]), H::pack2(y[k + 6], y[k + 7]));
                    } else if (mine) {
#pragma unroll
                        for (int k = 0; k < 16; k += 4)
                            *reinterpret_cast<float4 *>(left + j + k) = make_float4(y[k], y[k + 1], y[k + 2], y[k + 3]);
                    }
                }
                fence_before_sync();
                if (mine) {
                    if (!whole) p.plan.stats(blockIdx.x, x.part)[row] = make_float2(m - H::kShift, l);
                    else if (p.lse != nullptr)
                        p.lse[at] = ((m == kNone ? 0.f : m - H::kShift) + log2f(l)) * 0.69314718055994530942f;
                }
            }
            if (both) arrive(merged);
        }
        tmem_wait_st();  // (given up or not, TMEM is freed behind the stores)
    } else {
        regs_dec<kOtherRegs>();
        const uint32_t leader = elect_leader();
        if (warp == 8 || warp == 10) {
            // ================== loads: keys, or values ===================
            const bool values = warp == 10;
            const int boxes = KT / p.box;
            // This lane's box of a tile.  Its page is read a tile ahead.
            const int first = lane * p.box;
            int base = 0;                   // loads of the units so far, of both warps
            uint32_t mine = 0, parity = 0;  // stages that this warp has loaded last, and their phases
            Work x;
#pragma unroll 1
            for (int u = 0; next_unit(u, x); ++u) {
                const int32_t *table = p.page_table + (int64_t)x.b * p.max_pages;
                auto page_of = [&](int i) {
                    const int k = x.key0 + i * KT + first;
                    return i < x.n && lane < boxes && k + p.box > x.lo && k < x.hi ? table[(unsigned)k / (unsigned)p.page_size]
                                                                                   : -1;
                };
                int ahead = page_of(0);
#pragma unroll 1
                for (int i = 0; i < x.n; ++i) {
                    const int at = base + (values ? seq_v<MODE>(i, x.n) : seq_k<MODE>(i)), st = at % NS;
                    const int k0 = x.key0 + i * KT, k = k0 + first;
                    const int b0 = (max(x.lo, k0) - k0) / p.box, b1 = (min(x.hi - k0, KT) + p.box - 1) / p.box;
                    const int page = ahead;
                    ahead = page_of(i + 1);
                    if (at >= NS && !(ok = wait(&empty[st], at / NS - 1))) break;
                    since = globaltimer_lo();
                    if (leader) mbar_arrive_expect_tx(&full[st], (uint32_t)((b1 - b0) * p.box * 128 * NB));
                    __syncwarp();
                    mine |= 1u << st;
                    parity = (parity & ~(1u << st)) | ((uint32_t)(at / NS) & 1u) << st;
                    if (lane >= b0 && lane < b1) {
                        int index = p.none;  // (out of the tensor: zeros)
                        if (page >= 0 && page < p.num_pages) index = page * p.page_step + x.hk * p.head_step;
                        else atomicOr(p.err, (uint32_t)GDN_DEVERR_BAD_INDEX);
                        tma_load_5d(sm + L::oKv + st * L::kTile + first * 128 * NB, values ? &mv : &mk, 0, 0, 0,
                                    (int)((unsigned)k % (unsigned)p.page_size) >> 3, index, &full[st]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                base += 2 * x.n;
            }
            // The copies in flight land before the CTA ends, whoever gave up.  (To the end: the
            // last ones of both warps.  Given up: this warp's own; a stage that the other one
            // has filled since may take the wait its time.)
            __syncwarp();
#pragma unroll 1
            for (int y = 0; y < NS; ++y) {
                const int at = base - 1 - y;
                if (ok && at >= 0) mbar_wait(&full[at % NS], (uint32_t)(at / NS) & 1u, kDefaultWaitNs / 8);
                if (!ok && (mine >> y & 1)) mbar_wait(&full[y], parity >> y & 1, kDefaultWaitNs / 8);
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
                if (more) {
                    x = work_of<MODE>(p, w);
                    cut = w.cut(p, p.plan);
                }
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
                more = w.next(p, p.plan);
            }
            if (lane == 0) *p.plan.cut(blockIdx.x) = cut;
            // (a barrier's last completion: older ones are not told from none)
            for (int x = max(0, live - (MODE == kOne ? 2 : 1)); x < live; ++x)
                mbar_wait(&q_full[MODE == kOne ? x & 1 : 0], (uint32_t)(MODE == kOne ? x >> 1 : x) & 1u, kDefaultWaitNs / 8);
        } else {
            // ============================ MMAs ===========================
            // (a negative scale: of the scores' queries)
            const uint32_t id_s = idesc_f16(128, KT, false, false, H::kBf16) | (p.scale < 0.f ? 1u << 13 : 0u);
            const uint32_t id_o = idesc_f16(128, p.d, false, true, H::kBf16);
            const uint32_t s0 = smem_u32(sm);
            int base = 0, live = 0, items[2] = {0, 0};
            Work x;
#pragma unroll 1
            for (int u = 0; next_unit(u, x); ++u) {
                if (x.n == 0) continue;
                const int n = x.n, buf = MODE == kOne ? live & 1 : 0;
                if (!(ok = wait(&q_full[buf], MODE == kOne ? live >> 1 : live))) break;
                int k_seen = -1, v_seen = -1;
                // S of slot s = Q K_i^T; the tile goes back behind its last product
                auto scores = [&](int s, int i, bool last) {
                    const int at = base + seq_k<MODE>(i), st = at % NS;
                    if (i != k_seen && !(ok = wait(&full[st], at / NS))) return;
                    k_seen = i;
                    since = globaltimer_lo();
                    fence_after_sync();
                    const uint64_t qd = desc_sw128(s0 + (MODE == kOne ? buf : s) * L::kTile, 16, 1024);
                    const uint64_t kd = desc_sw128(s0 + L::oKv + st * L::kTile, 16, NB * 1024);
#pragma unroll
                    for (int k = 0; k < 4 * NB; ++k)
                        if (16 * k < p.d)
                            mma_f16_warp(leader, tm + tS + 128 * s, desc_add(qd, (k >> 2) * kBlock + (k & 3) * 32),
                                         desc_add(kd, (k >> 2) * 1024 + (k & 3) * 32), id_s, k > 0);
                    mma_commit_warp(leader, &s_full[s]);
                    if (last) mma_commit_warp(leader, &empty[st]);
                };
                // O of slot s += P V_i
                auto sums = [&](int s, int i, bool first, bool last, bool end) {
                    const int at = base + seq_v<MODE>(i, n), st = at % NS;
                    if (i != v_seen) {
                        if (!(ok = wait(&full[st], at / NS))) return;
                        // Values of keys that no query of the unit sees: zeros, whatever was
                        // there (their weights are 0, but 0 times NaN is not).
                        const int k0 = x.key0 + i * KT;
                        const int r0 = max(0, x.lo - k0), r1 = min(KT, x.hi - k0);
                        if (r0 > 0 || r1 < KT) {
                            uint8_t *v = sm + L::oKv + st * L::kTile;
#pragma unroll 1
                            for (int e = lane; e < (r0 + KT - r1) * 8 * NB; e += 32) {
                                int row = e / (8 * NB);
                                row = row < r0 ? row : row - r0 + r1;
                                *reinterpret_cast<uint4 *>(v + (row >> 3) * (NB * 1024) + (e / 8 % NB) * 1024 +
                                                           (row & 7) * 128 + (e & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
                            }
                            fence_proxy_async();
                            __syncwarp();
                        }
                        v_seen = i;
                    }
                    if (!(ok = wait(&p_ready[s], items[s]))) return;
                    ++items[s];
                    since = globaltimer_lo();
                    fence_after_sync();
                    const uint64_t vd = desc_sw128(s0 + L::oKv + st * L::kTile, 1024, NB * 1024);
#pragma unroll
                    for (int k = 0; k < KT / 16; ++k)
                        mma_f16_ta_warp(leader, tm + tO + 128 * s, tm + tS + 128 * s + 8 * k, desc_add(vd, k * NB * 2048),
                                        id_o, !first || k > 0);
                    if (last) mma_commit_warp(leader, &empty[st]);
                    if (end) mma_commit_warp(leader, &o_done[s]);
                };
                if constexpr (MODE == kPair) {
                    auto has = [&](int s, int i) { return i >= (s ? x.a[1] : x.a[0]) && i < (s ? x.e[1] : x.e[0]); };
                    // Turn y: sums of tile (y / 2) - 1 for slot y % 2, then its scores of the next
#pragma unroll 1
                    for (int y = 0; ok && y < 2 * n + 2; ++y) {
                        const int s = y & 1, i = (y >> 1) - 1;
                        if (has(s, i)) sums(s, i, !has(s, i - 1), s == 1 || !has(1, i), !has(s, i + 1));
                        if (ok && has(s, i + 1)) scores(s, i + 1, s == 1 || !has(1, i + 1));
                        // the unit's last scores are issued
                        if (ok && y == 2 * n - 1) mma_commit_warp(leader, q_free);
                    }
                } else {
                    // Turn y: sums of tile y - 2, then scores of tile y, for slot y % 2
#pragma unroll 1
                    for (int y = 0; ok && y < n + 2; ++y) {
                        const int s = y & 1, i = y - 2;
                        if (i >= 0) sums(s, i, i < 2, true, i >= n - 2);
                        if (ok && y < n) scores(s, y, true);
                        if (ok && y == n - 1) mma_commit_warp(leader, &q_free[buf]);
                    }
                }
                if (!ok) break;
                base += 2 * n;
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
    if (p.dt == GDN_F32 || p.page_size % 8 != 0 || p.num_pages == 0) return false;
    // tensor maps: addresses and strides of 16 bytes, strides below 2^40 bytes, indexes of 31 bits
    const uint64_t all = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k_pages) |
                         reinterpret_cast<uintptr_t>(p.v_pages) |
                         (uint64_t)(p.qs | p.page_stride | p.slot_stride | p.head_stride) * 2;
    if ((all & 15) != 0) return false;
    const int64_t limit = 1ll << 36;  // (a slot's stride is taken times 8)
    return p.qs < limit && p.page_stride < limit && p.slot_stride < limit && p.head_stride < limit &&
           steps_of(p).count < (1ll << 31) - 1;
}

Plan plan_tc(int B, int T, int Hq, int Hk, int d, bool varlen) {
    Plan s = plan_of(Hq, Hk, d, 128, sm_count_of_current_device());
    if (mean_tokens(B, T, varlen) > s.tokens) s.tokens *= 2;  // two blocks a unit
    return s;
}

cudaError_t launch_attention_tc(const AttentionParams &pp, const Plan &plan, cudaStream_t stream) {
    TcParams p{};
    static_cast<AttentionParams &>(p) = pp;
    p.plan = plan;
    p.slot_tokens = 128 / plan.gs;
    p.box = std::min(KT, p.page_size & -p.page_size);
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
    if (!encode_heads_map(&mq, p.q, bf, p.d, p.Hq, total, p.qs, plan.gs, p.slot_tokens) ||
        !encode_pages_map(&mk, p.k_pages, bf, p.d, p.page_size, p.slot_stride, x.count, x.unit, p.box) ||
        !encode_pages_map(&mv, p.v_pages, bf, p.d, p.page_size, p.slot_stride, x.count, x.unit, p.box))
        return cudaErrorInvalidValue;
    if (p.d == 128)
        return bf ? launch_nb<__nv_bfloat16, 2>(p, mq, mk, mv, stream) : launch_nb<__half, 2>(p, mq, mk, mv, stream);
    return bf ? launch_nb<__nv_bfloat16, 1>(p, mq, mk, mv, stream) : launch_nb<__half, 1>(p, mq, mk, mv, stream);
}

}  // namespace attn
}  // namespace gdn
