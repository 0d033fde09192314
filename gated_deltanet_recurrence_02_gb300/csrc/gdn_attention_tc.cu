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

#include "gdn_attention.cuh"

namespace gdn {
namespace attn {
namespace {

using namespace tc;

constexpr int KT = 128;           // keys of a tile
constexpr int kThreads = 384;     // two softmax warpgroups; a warp that loads, one that issues MMAs, two without work
// registers a thread: 168 at launch, of which the third warpgroup gives 96 to the others
constexpr int kSoftmaxRegs = 216, kOtherRegs = 72;
constexpr uint32_t kBlock = 16384;  // 128 rows of 64 elements
constexpr uint32_t tS = 0, tO = 256;  // TMEM: S (and P in its place) and O of a slot, 128 columns each
constexpr uint32_t kTmemCols = 512;
constexpr float kGrowth = 8.f;    // of the maximum's exponent, before O follows
constexpr int kAhead = 4;         // tiles of the next unit loaded before its queries

// Two ways to use the two slots (S and O in TMEM and a warpgroup each):
//  kPair   a unit has two blocks of up to 128 query rows, a slot each, which share the tiles
//  kOne    a unit has one block; the slots take its tiles in turn and are added up at the end
enum Mode { kPair, kOne };

template <int NB, int MODE>
struct Layout {
    static constexpr int kQ = 2;                           // blocks of queries in shared memory
    static constexpr uint32_t kTile = NB * kBlock;
    static constexpr int NS = NB == 2 ? 5 : 10;            // tiles of keys or values in flight
    static constexpr uint32_t oKv = kQ * kTile;
    static constexpr uint32_t oMerge = oKv + NS * kTile;   // [128] maxima and sums of slot 1 (kOne)
    static constexpr uint32_t oBar = oMerge + 1024;
    static constexpr uint32_t kSmem = oBar + 256 + 1024;   // + alignment slack
};

struct TcParams : AttentionParams {
    Plan plan;
    int G, slot_rows, slot_tokens;  // query heads a key head; query rows and tokens of a slot
    int box;                        // keys of a TMA box: the power of two in the page size
    float c;                        // |scale| log2 e
    bool negative;                  // scale < 0
};

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

// Tiles [a, e) of the unit that slot s works on, within the piece; rows of the slot.
struct SlotWork {
    int rows, a, e;
};
template <int MODE>
__device__ __forceinline__ SlotWork slot_work(const TcParams &p, const Walk &w, int s) {
    SlotWork x;
    const Unit &u = w.unit;
    const int rho0 = u.rho0 + (MODE == kPair ? s * p.slot_rows : 0);
    x.rows = max(0, min(p.slot_rows, u.rho1 - rho0));
    x.a = x.e = w.at.tile;
    if (x.rows == 0 || u.hi <= u.lo) return x;
    int lo = u.lo, hi = u.hi;
    if (MODE == kPair && p.causal) {
        const int t0 = rho0 / p.G, t1 = (rho0 + x.rows - 1) / p.G;
        hi = min(hi, w.row.first + t1 + 1);
        if (p.window > 0) lo = max(lo, w.row.first + t0 - p.window + 1);
        if (hi <= lo) return x;
    }
    x.a = max(w.at.tile, (lo - u.key0) / KT);
    x.e = max(x.a, min(w.end, (hi - u.key0 + KT - 1) / KT));
    return x;
}

template <typename E, int NB, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
attention_kernel(const TcParams p, const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv) {
    using H = Half16<E>;
    using L = Layout<NB, MODE>;
    constexpr int NS = L::NS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *sm = smem_align1k(smem_raw);
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::oBar), *empty = full + NS;
    uint64_t *q_full = empty + NS, *q_free = q_full + 2;     // of units in turn (kPair: the first of each)
    uint64_t *s_full = q_free + 2, *p_ready = s_full + 2, *o_done = p_ready + 2;  // a slot each
    uint64_t *other = o_done + 2, *merged = other + 1, *drain = other + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(other + 3);
    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const Plan &plan = p.plan;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
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
    const Place from = find_place<kThreads>(p, plan, p.G);
    fence_before_sync();
    __syncthreads();
    fence_after_sync();
    const uint32_t tm = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    bool ok = true;
    auto wait = [&](uint64_t *bar, int n) {  // for the n-th completion (from 0), a whole warp
        return __all_sync(0xffffffffu, mbar_wait(bar, (uint32_t)n & 1u, p.wait_ns)) != 0;
    };
    auto arrive = [&](uint64_t *bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    Walk w;
    bool more = w.start(p, plan, p.G, from);

    if (warp < 8) {
        // ============================ softmax ============================
        regs_inc<kSoftmaxRegs>();
        const int s = warp >> 2, r = (warp & 3) * 32 + lane;  // slot, row of the slot
        const uint32_t ts = tm + ((uint32_t)((warp & 3) * 32) << 16) + tS + 128 * s;
        const uint32_t to = tm + ((uint32_t)((warp & 3) * 32) << 16) + tO + 128 * s;
        float2 *merge = reinterpret_cast<float2 *>(sm + L::oMerge);
        const float2 c2 = make_float2(p.c, p.c);
        Cut cut{};
        int item = 0, done = 0, units = 0;
        for (; more; more = w.next(p, plan, p.G)) {
            const Unit &u = w.unit;
            const SlotWork x = slot_work<MODE>(p, w, s);
            const int rho = u.rho0 + (MODE == kPair ? s * p.slot_rows : 0) + r;
            const bool mine = r < x.rows;
            const bool idle = (warp & 3) * 32 >= x.rows;  // the whole warp has no row
            const int t = rho / p.G;
            int lo = 0, hi = 0x7fffffff;  // keys that the row sees (rows that are not there: any)
            if (mine) {
                hi = w.row.keys;
                if (p.causal) {
                    hi = min(hi, w.row.first + t + 1);
                    if (p.window > 0) lo = max(0, w.row.first + t - p.window + 1);
                }
            }
            float m = kNone, l = 0.f;  // m: c times the score that weights are relative to
            const int i0 = MODE == kPair ? x.a : x.a + s;
            for (int i = i0; i < x.e; i += MODE == kPair ? 1 : 2, ++item) {
                if (!(ok = wait(&s_full[s], item))) break;
                fence_after_sync();
                if (idle) {
                    arrive(&p_ready[s]);
                    continue;
                }
                uint32_t v[4][32];
#pragma unroll
                for (int g = 0; g < 4; ++g) tmem_ld32_async(ts + 32 * g, v[g]);
                tmem_wait_ld();
                if (p.negative)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[g][j] ^= 0x80000000u;
                const int a = lo - (u.key0 + i * KT), e = hi - (u.key0 + i * KT);
                if (__any_sync(0xffffffffu, a > 0 || e < KT)) {
#pragma unroll
                    for (int g = 0; g < 4; ++g)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (32 * g + j < a || 32 * g + j >= e) v[g][j] = 0xff800000u;
                }
                float top[4];
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    top[g] = __uint_as_float(v[g][0]);
#pragma unroll
                    for (int j = 1; j < 32; ++j) top[g] = fmaxf(top[g], __uint_as_float(v[g][j]));
                }
                const float now = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * p.c;
                const bool grow = now - m > kGrowth;  // (from none: always, unless there is still none)
                if (__any_sync(0xffffffffu, grow)) {
                    const float keep = grow ? ex2_approx(m - now) : 1.f;
                    m = grow ? now : m;
                    if (i != i0) {
                        // the slot's last product is done: S was issued behind it
                        l *= keep;
                        const float2 k2 = make_float2(keep, keep);
#pragma unroll
                        for (int g = 0; g < 4 * NB; ++g) {
                            if (16 * g < p.d) {
                                uint32_t o[16];
                                tmem_ld16_async(to + 16 * g, o);
                                tmem_wait_ld();
#pragma unroll
                                for (int j = 0; j < 16; j += 2) {
                                    const float2 y = __fmul2_rn(k2, make_float2(__uint_as_float(o[j]), __uint_as_float(o[j + 1])));
                                    o[j] = __float_as_uint(y.x);
                                    o[j + 1] = __float_as_uint(y.y);
                                }
                                tmem_st16(to + 16 * g, o);
                            }
                        }
                    }
                }
                // (held finite: without keys so far weights are 0)
                const float off = H::kShift - fmaxf(m, -3.4028235e38f);
                const float2 off2 = make_float2(off, off);
                float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    uint32_t pk[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        float2 y = __ffma2_rn(make_float2(__uint_as_float(v[g][j]), __uint_as_float(v[g][j + 1])), c2, off2);
                        y.x = ex2_approx(y.x);
                        y.y = ex2_approx(y.y);
                        sum[(j >> 1) & 1] = __fadd2_rn(sum[(j >> 1) & 1], y);
                        pk[j / 2] = H::pack2(y.x, y.y);
                    }
                    tmem_st16(ts + 16 * g, pk);
                }
                tmem_wait_st();
                fence_before_sync();
                arrive(&p_ready[s]);
                sum[0] = __fadd2_rn(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
            }
            if (!ok) break;
            const bool any = x.e > i0;  // the slot has sums of its own
            if (any) {
                if (!(ok = wait(&o_done[s], done))) break;
                ++done;
                fence_after_sync();
            }
            float f0 = 1.f, f1 = 0.f;  // factors of this slot's sums, and of the other's (kOne)
            bool both = false;
            if constexpr (MODE == kOne) {
                if (x.e - x.a > 1) {
                    if (s == 1) {
                        merge[r] = make_float2(m, l);
                        arrive(other);
                        // (the next unit's products here wait for what the others read)
                        if (!(ok = wait(merged, units))) break;
                    } else {
                        if (!(ok = wait(other, units))) break;
                        fence_after_sync();
                        const float2 ml = merge[r];
                        const float top = fmaxf(m, ml.x), safe = top == kNone ? 0.f : top;
                        f0 = ex2_approx(m - safe);
                        f1 = ex2_approx(ml.x - safe);
                        m = top;
                        l = f0 * l + f1 * ml.y;
                        both = true;
                    }
                    ++units;
                }
            }
            const bool writes = MODE == kPair || s == 0;
            if (writes && !idle) {
                const bool whole = w.whole();
                const float inv = !whole ? 1.f : l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // (a NaN stays one)
                const long at = (w.row.tok0 + t) * p.Hq + w.at.hk * p.G + (rho - t * p.G);
                E *out = reinterpret_cast<E *>(p.out) + at * p.d;
                float *part = plan.sums(blockIdx.x, w.part()) + (size_t)(rho - u.rho0) * p.d;
                if (!any) f0 = 0.f;
#pragma unroll 1
                for (int g = 0; 16 * g < p.d; ++g) {
                    uint32_t o[16], o1[16];
                    float y[16];
                    if (any) tmem_ld16_async(to + 16 * g, o);
                    if (both) tmem_ld16_async(to + 128 + 16 * g, o1);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        y[j] = any ? __uint_as_float(o[j]) * (f0 * inv) : 0.f;
                        if (both) y[j] = fmaf(__uint_as_float(o1[j]), f1 * inv, y[j]);
                    }
                    if (mine && whole) {
#pragma unroll
                        for (int j = 0; j < 16; j += 8)
                            *reinterpret_cast<uint4 *>(out + 16 * g + j) =
                                make_uint4(H::pack2(y[j], y[j + 1]), H::pack2(y[j + 2], y[j + 3]),
                                           H::pack2(y[j + 4], y[j + 5]), H::pack2(y[j + 6], y[j + 7]));
                    } else if (mine) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4)
                            *reinterpret_cast<float4 *>(part + 16 * g + j) = make_float4(y[j], y[j + 1], y[j + 2], y[j + 3]);
                    }
                }
                fence_before_sync();
                if (mine) {
                    if (!whole) plan.stats(blockIdx.x, w.part())[rho - u.rho0] = make_float2(m - H::kShift, l);
                    else if (p.lse != nullptr)
                        p.lse[at] = ((m == kNone ? 0.f : m - H::kShift) + log2f(l)) * 0.69314718055994530942f;
                }
            }
            if constexpr (MODE == kOne)
                if (both) arrive(merged);
            if (w.at.tile > 0) cut.head = w.end == u.tiles ? 1 : 2;
            else if (w.end < u.tiles) cut.tail = 1, cut.b = w.at.b, cut.hk = w.at.hk, cut.block = w.at.block;
        }
        if (threadIdx.x == 0) *plan.cut(blockIdx.x) = cut;
        tmem_wait_st();  // (given up or not, TMEM is freed behind the stores)
    } else {
      regs_dec<kOtherRegs>();
      if (warp == 8) {
        // ============================= loads =============================
        const uint32_t leader = elect_leader();
        const int boxes = KT / p.box;
        const uint32_t q_bytes = (uint32_t)p.slot_rows * 128 * NB;
        int base = 0, units = 0;  // loads and units so far
        for (; more; more = w.next(p, plan, p.G)) {
            const Unit &u = w.unit;
            if (u.hi <= u.lo) continue;
            const int n = w.end - w.at.tile;
            auto queries = [&]() {
                // (kOne: two blocks in turn; kPair: both for one unit)
                const int buf = MODE == kOne ? units & 1 : 0, turn = MODE == kOne ? units >> 1 : units;
                if (turn > 0 && !(ok = wait(&q_free[buf], turn - 1))) return;
                if (leader) {
                    const int slots = MODE == kPair ? 2 : 1;
                    mbar_arrive_expect_tx(&q_full[buf], q_bytes * slots);
                    for (int s = 0; s < slots; ++s)
                        for (int j = 0; j < NB; ++j)
                            tma_load_3d(sm + (buf + s) * L::kTile + j * kBlock, &mq, 64 * j, w.at.hk * p.G,
                                        (int)(w.row.tok0 + u.rho0 / p.G + s * p.slot_tokens), &q_full[buf]);
                }
                __syncwarp();
            };
            const int q_at = units == 0 ? 0 : min(kAhead, 2 * n - 1);
            for (int x = 0; ok && x < 2 * n; ++x) {
                if (x == q_at) queries();
                if (!ok) break;
                // the x-th load: keys or values of tile i
                bool values;
                int i;
                if (MODE == kPair) values = x & 1, i = x >> 1;
                else if (x == 2 * n - 1) values = true, i = n - 1;
                else values = x > 0 && (x & 1) == 0, i = values ? x / 2 - 1 : (x + 1) / 2;
                const int at = base + x, st = at % NS;
                const int k0 = u.key0 + (w.at.tile + i) * KT;
                const int b0 = max(0, u.lo - k0) / p.box, b1 = (min(u.hi - k0, KT) + p.box - 1) / p.box;
                // this lane's boxes: box (lane % boxes), block (lane / boxes) and so on
                const int box = lane & (boxes - 1);
                int page = 0, slot0 = 0;
                const bool there = box >= b0 && box < b1;
                if (there) {
                    const int k = k0 + box * p.box;
                    const int pg = k / p.page_size;
                    slot0 = k - pg * p.page_size;
                    page = p.page_table[(int64_t)w.at.b * p.max_pages + pg];
                    if (page < 0 || page >= p.num_pages) {
                        atomicOr(p.err, (uint32_t)GDN_DEVERR_BAD_INDEX);
                        page = p.num_pages;  // (out of the tensor: zeros)
                    }
                }
                if (at >= NS && !(ok = wait(&empty[st], at / NS - 1))) break;
                if (leader) mbar_arrive_expect_tx(&full[st], (uint32_t)((b1 - b0) * p.box * 128 * NB));
                __syncwarp();
                uint8_t *dst = sm + L::oKv + st * L::kTile + box * p.box * 128;
                if (there)
                    for (int j = lane / boxes; j < NB; j += 32 / boxes)
                        tma_load_4d(dst + j * kBlock, values ? &mv : &mk, 64 * j, slot0, w.at.hk, page, &full[st]);
                __syncwarp();
            }
            if (!ok) break;
            base += 2 * n;
            ++units;
        }
        // The copies in flight land before the CTA ends, whoever gave up.
        __syncwarp();
        for (int x = max(0, base - NS); x < base; ++x) mbar_wait(&full[x % NS], (uint32_t)(x / NS) & 1u, kDefaultWaitNs / 8);
        // (a barrier's last completion: older ones are not told from none)
        for (int x = max(0, units - (MODE == kOne ? 2 : 1)); x < units; ++x)
            mbar_wait(&q_full[MODE == kOne ? x & 1 : 0], (uint32_t)(MODE == kOne ? x >> 1 : x) & 1u, kDefaultWaitNs / 8);
      } else if (warp == 9) {
        // ============================== MMAs =============================
        const uint32_t leader = elect_leader();
        const uint32_t id_s = idesc_f16(128, KT, false, false, H::kBf16), id_o = idesc_f16(128, p.d, false, true, H::kBf16);
        const uint32_t s0 = smem_u32(sm);
        int base = 0, units = 0, items[2] = {0, 0};
        for (; more; more = w.next(p, plan, p.G)) {
            const Unit &u = w.unit;
            if (u.hi <= u.lo) continue;
            const int n = w.end - w.at.tile;
            SlotWork x[2];
            if (MODE == kPair)
                for (int s = 0; s < 2; ++s) {
                    x[s] = slot_work<MODE>(p, w, s);
                    x[s].a -= w.at.tile;
                    x[s].e -= w.at.tile;
                }
            const int buf = MODE == kOne ? units & 1 : 0;
            if (!(ok = wait(&q_full[buf], MODE == kOne ? units >> 1 : units))) break;
            int k_seen = -1, v_seen = -1;
            // S of slot s = Q K_i^T; the tile goes back behind its last product
            auto scores = [&](int s, int i, bool last) {
                const int at = base + seq_k<MODE>(i), st = at % NS;
                if (i != k_seen && !(ok = wait(&full[st], at / NS))) return;
                k_seen = i;
                fence_after_sync();
                const uint64_t qd = desc_sw128(s0 + (MODE == kOne ? buf : s) * L::kTile, 16, 1024);
                const uint64_t kd = desc_sw128(s0 + L::oKv + st * L::kTile, 16, 1024);
#pragma unroll
                for (int k = 0; k < 4 * NB; ++k)
                    if (16 * k < p.d) {
                        const uint32_t off = (k >> 2) * kBlock + (k & 3) * 32;
                        mma_f16_warp(leader, tm + tS + 128 * s, desc_add(qd, off), desc_add(kd, off), id_s, k > 0);
                    }
                mma_commit_warp(leader, &s_full[s]);
                if (last) mma_commit_warp(leader, &empty[st]);
            };
            // O of slot s += P V_i
            auto sums = [&](int s, int i, bool first, bool last, bool end) {
                const int at = base + seq_v<MODE>(i, n), st = at % NS;
                if (i != v_seen) {
                    if (!(ok = wait(&full[st], at / NS))) return;
                    // Values of keys that no query of the unit sees: zeros, whatever was there
                    // (their weights are 0, but 0 times NaN is not).
                    const int k0 = u.key0 + (w.at.tile + i) * KT;
                    const int r0 = max(0, u.lo - k0), r1 = min(KT, u.hi - k0);
                    if (r0 > 0 || r1 < KT) {
                        uint8_t *v = sm + L::oKv + st * L::kTile;
                        for (int e = lane; e < (r0 + KT - r1) * 8 * NB; e += 32) {
                            const int q = e & 7, row = (e >> 3) / NB, j = (e >> 3) - row * NB;
                            *reinterpret_cast<uint4 *>(v + j * kBlock + (row < r0 ? row : row - r0 + r1) * 128 + q * 16) =
                                make_uint4(0u, 0u, 0u, 0u);
                        }
                        fence_proxy_async();
                        __syncwarp();
                    }
                    v_seen = i;
                }
                if (!(ok = wait(&p_ready[s], items[s]))) return;
                ++items[s];
                fence_after_sync();
                const uint64_t vd = desc_sw128(s0 + L::oKv + st * L::kTile, kBlock, 1024);
#pragma unroll
                for (int k = 0; k < KT / 16; ++k)
                    mma_f16_ta_warp(leader, tm + tO + 128 * s, tm + tS + 128 * s + 8 * k, desc_add(vd, k * 2048), id_o,
                                    !first || k > 0);
                if (last) mma_commit_warp(leader, &empty[st]);
                if (end) mma_commit_warp(leader, &o_done[s]);
            };
            if constexpr (MODE == kPair) {
                auto has = [&](int s, int i) { return i >= x[s].a && i < x[s].e; };
                auto next = [&](int s, int i) {  // scores of tile i for slot s, if it has one
                    if (ok && has(s, i)) scores(s, i, s == 1 || !has(1, i));
                };
                next(0, 0);
                next(1, 0);
                for (int i = 0; ok && i < n; ++i)
                    for (int s = 0; ok && s < 2; ++s) {
                        if (has(s, i)) sums(s, i, i == x[s].a, s == 1 || !has(1, i), i == x[s].e - 1);
                        next(s, i + 1);
                        // the unit's last scores are issued
                        if (ok && s == 1 && i == n - 2) mma_commit_warp(leader, &q_free[0]);
                    }
                if (ok && n == 1) mma_commit_warp(leader, &q_free[0]);
            } else {
                scores(0, 0, true);
                if (ok && n > 1) scores(1, 1, true);
                if (ok && n <= 2) mma_commit_warp(leader, &q_free[buf]);
                for (int i = 0; ok && i < n; ++i) {
                    sums(i & 1, i, i < 2, true, i >= n - 2);
                    if (ok && i + 2 < n) {
                        scores(i & 1, i + 2, true);
                        if (ok && i + 3 == n) mma_commit_warp(leader, &q_free[buf]);
                    }
                }
            }
            if (!ok) break;
            base += 2 * n;
            ++units;
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
    constexpr uint32_t bytes = Layout<NB, MODE>::kSmem;
    cudaError_t e = set_smem_once<attention_kernel<E, NB, MODE>>((int)bytes);
    if (e != cudaSuccess) return e;
    attention_kernel<E, NB, MODE><<<p.plan.ctas, kThreads, bytes, stream>>>(p, mq, mk, mv);
    e = cudaGetLastError();
    return e != cudaSuccess ? e : launch_join(p, p.plan, stream);
}

template <typename E, int NB>
cudaError_t launch_nb(const TcParams &p, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                      cudaStream_t stream) {
    return p.plan.rows > p.slot_rows ? launch_mode<E, NB, kPair>(p, mq, mk, mv, stream)
                                     : launch_mode<E, NB, kOne>(p, mq, mk, mv, stream);
}

}  // namespace

bool tc_takes(const AttentionParams &p) {
    if (p.dt == GDN_F32 || p.Hq / p.Hk > 128 || p.page_size % 8 != 0 || p.num_pages == 0) return false;
    // tensor maps: addresses and strides of 16 bytes, strides below 2^40 bytes
    const uint64_t all = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k_pages) |
                         reinterpret_cast<uintptr_t>(p.v_pages) |
                         (uint64_t)(p.qs | p.page_stride | p.slot_stride | p.head_stride) * 2;
    if ((all & 15) != 0) return false;
    const int64_t limit = 1ll << 39;
    return p.qs < limit && p.page_stride < limit && p.slot_stride < limit && p.head_stride < limit;
}

Plan plan_tc(int B, int T, int Hq, int Hk, int d, bool varlen) {
    const int G = Hq / Hk, slot = G <= 128 ? 128 / G * G : G;
    const long mean = varlen ? ((long)T + B - 1) / std::max(B, 1) : T;
    Plan s{};
    s.rows = mean * G <= slot ? slot : 2 * slot;
    s.keys = KT;
    s.ctas = sm_count_of_current_device();
    s.d = d;
    return s;
}

cudaError_t launch_attention_tc(const AttentionParams &pp, const Plan &plan, cudaStream_t stream) {
    TcParams p{};
    static_cast<AttentionParams &>(p) = pp;
    p.plan = plan;
    p.G = p.Hq / p.Hk;
    p.slot_tokens = 128 / p.G;
    p.slot_rows = p.slot_tokens * p.G;
    p.box = std::min(KT, p.page_size & -p.page_size);
    p.negative = p.scale < 0.f;
    // (a scale of 0 gives every key that is seen the same weight, and -infinity still none)
    p.c = std::max(std::abs(p.scale) * kLog2e, 0x1p-126f);
    const long total = p.cu_seqlens != nullptr ? (long)p.T : (long)p.B * p.T;
    const bool bf = p.dt == GDN_BF16;
    CUtensorMap mq, mk, mv;
    if (!encode_heads_map(&mq, p.q, bf, p.d, p.Hq, total, p.d, p.qs, p.G, p.slot_tokens) ||
        !encode_pages_map(&mk, p.k_pages, bf, p.d, p.page_size, p.Hk, p.num_pages, p.slot_stride, p.head_stride,
                          p.page_stride, p.box) ||
        !encode_pages_map(&mv, p.v_pages, bf, p.d, p.page_size, p.Hk, p.num_pages, p.slot_stride, p.head_stride,
                          p.page_stride, p.box))
        return cudaErrorInvalidValue;
    if (p.d == 128)
        return bf ? launch_nb<__nv_bfloat16, 2>(p, mq, mk, mv, stream) : launch_nb<__half, 2>(p, mq, mk, mv, stream);
    return bf ? launch_nb<__nv_bfloat16, 1>(p, mq, mk, mv, stream) : launch_nb<__half, 1>(p, mq, mk, mv, stream);
}

}  // namespace attn
}  // namespace gdn
