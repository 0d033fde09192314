// gdn_attention.cuh -- how the attention kernels cut their work, and join what they cut.
//
// A unit is (row b, group of query heads that share a key head, block of tokens): its query
// rows are rho = t gs + g, gs heads a token, so that all of them read a tile of keys once.
// All units' tiles in a row, in the order of b, group, block, each unit with a few more in
// front for what it costs to begin and end, are cut into equal pieces, one a CTA, so that no
// lengths, however ragged, leave CTAs idle.  Lengths are on the device, so
// each CTA finds its piece there: a sum over the rows and a search along the one it starts
// in.  A unit that a cut goes through leaves its parts (unscaled sums, maxima, sums of
// weights) in the workspace, at most two a CTA: the end of a unit that an earlier CTA began
// (part 0) and the start of one that a later CTA goes on with (part 1).  The join, a second
// kernel, adds the parts up in the order of the keys, so the result does not depend on timing.
// (16 prompts of 200 to 2000 tokens, 4 of 32 heads, d = 64: 240 us with units counted by their
// tiles alone, 199 with what begins and ends them.)
#pragma once

#include "gdn_internal.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace attn {

constexpr float kNone = -INFINITY;
constexpr unsigned kAll = 0xffffffffu;

// What a CTA leaves for the join: the unit that it begins and does not end.
struct alignas(16) Cut {
    long row0;   // out row (token times Hq plus head) of its first query
    int tokens;  // 0: there is none
    int heads;   // that the group has (up to gs)
    int parts;   // CTAs that have a part of it, this one first
    int pad[3];
};

// The cutting, with the workspace's layout: Cut [ctas], maxima and sums [ctas][2][rows][2],
// sums [ctas][2][rows][d].
struct Plan {
    int tokens, gs;      // tokens of a unit, query heads of a group
    int per_key, G;      // groups, and query heads, of a key head
    int over;            // tiles that a unit's beginning and end cost
    int least_log2;      // tiles of a piece, the least
    int ctas, d;
    uint8_t *ws;
    __host__ __device__ int rows() const { return tokens * gs; }
    __host__ __device__ Cut *cut(int c) const { return reinterpret_cast<Cut *>(ws) + c; }
    __host__ __device__ float2 *stats(int c, int part) const {
        return reinterpret_cast<float2 *>(ws + (size_t)ctas * sizeof(Cut)) + ((size_t)c * 2 + part) * rows();
    }
    __host__ __device__ float *sums(int c, int part) const {
        return reinterpret_cast<float *>(ws + (size_t)ctas * (sizeof(Cut) + 2 * rows() * sizeof(float2))) +
               ((size_t)c * 2 + part) * rows() * d;
    }
    size_t bytes() const {
        return (size_t)ctas * (sizeof(Cut) + 2 * (size_t)rows() * (sizeof(float2) + d * sizeof(float)));
    }
};

// A row's tokens, and its keys as far as the page table has room for them.
struct Row {
    long tok0;
    int tokens, keys;
    int first;  // cache position of the first token (negative where there are more tokens than keys)
};

__device__ __forceinline__ Row row_at(const AttentionParams &p, int b) {
    Row r;
    row_range(p.cu_seqlens, b, p.T, r.tok0, r.tokens);
    const int len = max(p.kv_lens[b], 0);
    // (sums of a key's number and a tile's size stay below 2^31)
    const long room = min((long)p.max_pages * p.page_size, 0x7fffff00l);
    r.keys = len < room ? len : (int)room;
    r.first = len - r.tokens;
    return r;
}
// The first key that the window of a query at position `at` leaves it (before the first
// position, where a query has no keys at all: no sum here passes 32 bits).
__device__ __forceinline__ int window_start(const AttentionParams &p, int at) {
    return p.causal && p.window > 0 ? max(0, max(0, at) - p.window + 1) : 0;
}
__device__ __forceinline__ Row row_of_lane(const Row &r, int lane) {
    return Row{__shfl_sync(kAll, r.tok0, lane), __shfl_sync(kAll, r.tokens, lane), __shfl_sync(kAll, r.keys, lane),
               __shfl_sync(kAll, r.first, lane)};
}

// One unit's tokens and keys; tiles of KT keys.
struct Unit {
    int t0, t1;       // tokens
    int lo, hi;       // keys that any of them sees
    int key0, tiles;  // the first tile's first key, tiles (one at least)
};

template <int KT>
__device__ __forceinline__ Unit unit_of(const AttentionParams &p, const Plan &s, const Row &r, int block) {
    Unit u;
    u.t0 = block * s.tokens;
    u.t1 = min(u.t0 + s.tokens, r.tokens);
    u.lo = window_start(p, r.first + u.t0);
    u.hi = r.keys;
    if (p.causal) u.hi = min(u.hi, r.first + u.t1);
    u.key0 = u.lo & -KT;
    u.tiles = u.hi > u.lo ? (u.hi - u.key0 + KT - 1) / KT : 1;
    return u;
}

__device__ __forceinline__ int blocks_of(const Plan &s, const Row &r) {
    return (int)((unsigned)(r.tokens + s.tokens - 1) / (unsigned)s.tokens);
}

// A place in the order of all tiles, and the tiles from there to the CTA's end; the other
// pieces are `each` long, and one more before CTA `more`.
struct Place {
    int b, group, block, tile;
    long left, each, more;
    Row row;  // of b
};

// Where this CTA's piece starts.  Each warp sums up a stretch of the rows, 32 rows at a time;
// where rows have many blocks, the lanes share each row's.  (One thread a row took 3 us for
// every 60 blocks of the longest.)  Called by all THREADS threads.
template <int KT, int THREADS>
__device__ Place find_place(const AttentionParams &p, const Plan &s) {
    constexpr int kWarps = THREADS / 32;
    __shared__ long sums[kWarps];
    __shared__ Place found;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, groups = p.Hk * s.per_key;
    const int per = (p.B + kWarps - 1) / kWarps;
    const int b0 = min(warp * per, p.B), b1 = min(b0 + per, p.B);
    // inclusive sums over the lanes
    auto scan = [&](long x) {
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const long y = __shfl_up_sync(kAll, x, o);
            if (lane >= o) x += y;
        }
        return x;
    };
    if (threadIdx.x == 0) found.left = 0;
    // Two passes over the rows, 32 a time: what they come to, and (by the warp that has the
    // piece's start) where that is.  Each in the same code: a launch finds the instruction
    // cache empty, and waits for every line of it.
    Row mine{0, 0, 0, 0};  // of lane b % 32
    long n = 0, all = 0, rest = -1, left = 0, each = 0, more = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int b = b0; b < b1; b += 32) {
            if (pass == 0 || b1 - b0 > 32) {
                // tiles of 32 rows from b on for one group, a lane each
                mine = b + lane < b1 ? row_at(p, b + lane) : Row{0, 0, 0, 0};
                const int blocks = blocks_of(s, mine);
                unsigned some = __ballot_sync(kAll, blocks > 0);
                const bool wide = __any_sync(kAll, blocks > 4);  // the lanes share each row's blocks
                n = 0;
                do {
                    const int x = wide ? __ffs(some) - 1 : lane;
                    const Row r = row_of_lane(mine, max(x, 0));
                    const int its = __shfl_sync(kAll, blocks, max(x, 0));
                    long part = 0;
#pragma unroll 1
                    for (int i = wide ? lane : 0; i < its; i += wide ? 32 : 1) part += unit_of<KT>(p, s, r, i).tiles + s.over;
                    if (wide) {
#pragma unroll 1
                        for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(kAll, part, o);
                    }
                    if (!wide || lane == x) n = part;
                    some &= some - 1;
                } while (wide && some != 0);
            }
            const long upto = scan(n * groups);
            if (pass == 0) {
                all += __shfl_sync(kAll, upto, 31);
                continue;
            }
            const unsigned in = __ballot_sync(kAll, rest < upto);
            if (in == 0) {
                rest -= __shfl_sync(kAll, upto, 31);
                continue;
            }
            const int x = __ffs(in) - 1;
            const long of_row = __shfl_sync(kAll, n, x);
            rest -= __shfl_sync(kAll, upto, x) - of_row * groups;
            const Row r = row_of_lane(mine, x);
            int group = 0, block = 0;
            if (groups > 1) {
                group = (rest | of_row) >> 31 ? (int)(rest / of_row) : (int)((unsigned)rest / (unsigned)of_row);
                rest -= group * of_row;
            }
            const int blocks = blocks_of(s, r);
            if (blocks > 1) {
#pragma unroll 1
                for (int i = 0;; i += 32) {
                    const int t = i + lane < blocks ? unit_of<KT>(p, s, r, i + lane).tiles + s.over : 0;
                    const long sum = scan(t);
                    const unsigned at = __ballot_sync(kAll, rest < sum);
                    if (at == 0) {
                        rest -= __shfl_sync(kAll, sum, 31);
                        continue;
                    }
                    const int y = __ffs(at) - 1;
                    rest -= __shfl_sync(kAll, sum - t, y);
                    block = i + y;
                    break;
                }
            }
            // (in what a unit has in front: at its first tile, the rest of that gone)
            const int ahead = max(0, s.over - (int)min(rest, 1l << 30));
            if (lane == 0) found = Place{b + x, group, block, (int)max(0l, rest - s.over), left - ahead, each, more, r};
            break;
        }
        if (pass == 1) break;
        if (lane == 0) sums[warp] = all;
        __syncthreads();
        long before = 0, total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const long x = sums[w];
            if (w < warp) before += x;
            total += x;
        }
        // Equal pieces of at least 2^least_log2, the first ones a tile longer
        const int c = blockIdx.x;
        const int n_ctas = (int)min((long)s.ctas, max(1l, total >> s.least_log2));
        each = total >> 31 ? total / n_ctas : (long)((unsigned)total / (unsigned)n_ctas);
        more = total - each * n_ctas;
        left = c < n_ctas ? each + (c < more ? 1 : 0) : 0;
        rest = each * c + min((long)c, more) - before;
        if (left <= 0 || rest < 0 || rest >= all) break;
    }
    __syncthreads();
    return found;
}

// The piece's units one after another: of the unit at hand the tiles [at.tile, end).
template <int KT>
struct Walk {
    Place at;
    Row row;
    Unit unit;
    int end, blocks;
    __device__ __forceinline__ void load(const AttentionParams &p, const Plan &s) {
        unit = unit_of<KT>(p, s, row, at.block);
        end = (int)min((long)unit.tiles, at.tile + at.left);
    }
    __device__ __forceinline__ bool start(const AttentionParams &p, const Plan &s, const Place &from) {
        at = from;
        if (at.left <= 0) return false;
        row = at.row;
        blocks = blocks_of(s, row);
        load(p, s);
        return true;
    }
    __device__ __forceinline__ bool next(const AttentionParams &p, const Plan &s) {
        at.left -= end - at.tile + s.over;
        if (at.left <= 0) return false;
        at.tile = 0;
        if (++at.block == blocks) {
            at.block = 0;
            if (++at.group == p.Hk * s.per_key) {
                at.group = 0;
                do {
                    if (++at.b >= p.B) return false;
                    row = row_at(p, at.b);
                    blocks = blocks_of(s, row);
                } while (blocks == 0);
            }
        }
        load(p, s);
        return true;
    }
    // 0, 1: the CTA's part that the cut unit leaves; -1: the unit is whole.
    __device__ __forceinline__ int part() const { return at.tile > 0 ? 0 : end < unit.tiles ? 1 : -1; }
    __device__ __forceinline__ int key_head(const Plan &s) const { return s.per_key == 1 ? at.group : at.group / s.per_key; }
    // First query head of the group, and its heads.
    __device__ __forceinline__ int head0(const AttentionParams &p, const Plan &s) const {
        const int k = key_head(s);
        return k * s.G + (at.group - k * s.per_key) * s.gs;
    }
    __device__ __forceinline__ int heads(const AttentionParams &p, const Plan &s) const {
        return min(s.gs, (key_head(s) + 1) * s.G - head0(p, s));
    }
    // What the CTA leaves for the join, after its last unit (one thread).
    __device__ __forceinline__ Cut cut(const AttentionParams &p, const Plan &s) const {
        Cut c{};
        if (part() != 1) return c;
        c.row0 = (row.tok0 + unit.t0) * p.Hq + head0(p, s);
        c.tokens = unit.t1 - unit.t0;
        c.heads = heads(p, s);
        // CTAs from here on: pieces of each + 1 tiles up to CTA `more`, then of each (all of
        // them the unit's tiles)
        const long rest = unit.tiles - end, longer = max(0l, at.more - (long)(blockIdx.x + 1));
        const long in = longer * (at.each + 1);
        c.parts = 1 + (int)(rest <= in ? (rest + at.each) / (at.each + 1) : longer + (rest - in + at.each - 1) / at.each);
        return c;
    }
};

// Joins the parts of cut units; maxima are those of scores times log2 e.  Grid (ctas, slices):
// CTA x takes the unit that CTA x of the attention began and did not end, a warp four query
// rows at a time (eight parts each a look: most units have two), so that all their loads are
// on their way together; D / 32 columns a lane.
//
// SHARE: of no more than 16 rows two to eight warps share the parts and are added up in order
// through shared memory, for a single token over a long cache leaves few rows and many parts
// (8000 keys, 4 of 16 heads, d = 128: the whole call 24 us with one warp for a row's parts, 16
// so; 30000 keys 30 and 20).  Not for other calls: with shared memory the join's CTAs no longer
// start next to the attention's (3 rows of up to 65 tokens, fp32: 22 us, without it 16).
template <typename T, int D, bool SHARE>
__global__ void __launch_bounds__(256) join_kernel(const AttentionParams p, const Plan s) {
    constexpr int kRows = 4, kLook = 32 / kRows, W = D / 32, kWarps = 8;
    struct alignas(4 * W) Cols {
        float v[W];
    };
    __shared__ Cols shared[SHARE ? kWarps : 1][kRows][32];
    __shared__ float shared_sum[SHARE ? kWarps : 1][kRows];
    tc::grid_dependency_wait();
    const Cut c = *s.cut(blockIdx.x);
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, n = c.tokens * s.gs;
    // Warps that share four rows' parts (then all rows are had in one turn)
    const int split = !SHARE || c.parts <= kLook ? 1 : n <= 4 ? 8 : n <= 8 ? 4 : n <= 16 ? 2 : 1;
    if (split > 1 && blockIdx.y > 0) return;
    const int share = warp % split, per = (c.parts + split - 1) / split;
    const int x_begin = share * per, x_end = min(c.parts, x_begin + per);
    const int first = (blockIdx.y * kWarps + warp) / split * kRows, step = gridDim.y * kWarps * kRows;
    for (int i0 = first; i0 < (split > 1 ? first + 1 : n); i0 += step) {
        const int mine = min(i0 + lane / kLook, n - 1);  // the row whose statistics the lane reads
        auto stats = [&](int x) {
            x += lane % kLook;
            return x < c.parts ? s.stats(blockIdx.x + x, x == 0)[mine] : make_float2(kNone, 0.f);
        };
        auto over = [&](float x, auto f) {  // over the lanes of a row
            for (int o = kLook / 2; o > 0; o >>= 1) x = f(x, __shfl_xor_sync(kAll, x, o));
            return x;
        };
        const float2 ml0 = stats(0);
        float top = ml0.x;
#pragma unroll 4
        for (int x = kLook; x < c.parts; x += kLook) top = fmaxf(top, stats(x).x);
        top = over(top, [](float a, float b) { return fmaxf(a, b); });
        const float safe = top == kNone ? 0.f : top;
        float sum = 0.f, acc[kRows][W];
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
            for (int e = 0; e < W; ++e) acc[r][e] = 0.f;
        for (int x0 = x_begin; x0 < x_end; x0 += kLook) {
            float2 ml = x0 == 0 ? ml0 : stats(x0);
            if (x0 + lane % kLook >= x_end) ml = make_float2(kNone, 0.f);
            const float weight = exp2f(ml.x - safe);
            sum = fmaf(weight, ml.y, sum);
#pragma unroll 4
            for (int x = x0; x < min(x_end, x0 + kLook); ++x) {
                Cols v[kRows];
#pragma unroll
                for (int r = 0; r < kRows; ++r)
                    v[r] = *reinterpret_cast<const Cols *>(s.sums(blockIdx.x + x, x == 0) +
                                                           (size_t)min(i0 + r, n - 1) * D + lane * W);
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const float w = __shfl_sync(kAll, weight, r * kLook + x - x0);
#pragma unroll
                    for (int e = 0; e < W; ++e) acc[r][e] = fmaf(w, v[r].v[e], acc[r][e]);
                }
            }
        }
        sum = over(sum, [](float a, float b) { return a + b; });
        if (SHARE && split > 1) {
            if (share > 0) {
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
#pragma unroll
                    for (int e = 0; e < W; ++e) shared[warp][r][lane].v[e] = acc[r][e];
                }
                if (lane % kLook == 0) shared_sum[warp][lane / kLook] = sum;
            }
            __syncthreads();
            if (share > 0) break;
            for (int y = warp + 1; y < warp + split; ++y) {
#pragma unroll
                for (int r = 0; r < kRows; ++r)
#pragma unroll
                    for (int e = 0; e < W; ++e) acc[r][e] += shared[y][r][lane].v[e];
                sum += shared_sum[y][lane / kLook];
            }
        }
        const float lse = (safe + log2f(sum)) * 0.69314718055994530942f;
        const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;  // (a NaN stays one)
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const float f = __shfl_sync(kAll, inv, r * kLook), log_sum = __shfl_sync(kAll, lse, r * kLook);
            const int i = i0 + r, t = i / s.gs, g = i - t * s.gs;
            if (i >= n || g >= c.heads) continue;
            const long at = c.row0 + (long)t * p.Hq + g;
            struct alignas(sizeof(T) * W) Out {
                T v[W];
            } out;
#pragma unroll
            for (int e = 0; e < W; ++e) st_out(&out.v[e], acc[r][e] * f);
            *reinterpret_cast<Out *>(reinterpret_cast<T *>(p.out) + at * D + lane * W) = out;
            if (p.lse != nullptr && lane == 0) p.lse[at] = log_sum;
        }
    }
}

// Launched behind an attention kernel, while it still runs, which hides the launch.  (Its CTAs
// start where that one's have left: a CTA of the tensor-core kernel has all registers.)
cudaError_t launch_join(const AttentionParams &p, const Plan &s, cudaStream_t stream);

// Units of up to `rows` query rows.
inline Plan plan_of(int Hq, int Hk, int d, int rows, int ctas, int over, int least_log2) {
    Plan s{};
    s.G = Hq / Hk;
    s.per_key = (s.G + rows - 1) / rows;
    s.gs = (s.G + s.per_key - 1) / s.per_key;
    s.tokens = rows / s.gs;
    s.over = over;
    s.least_log2 = least_log2;
    s.ctas = ctas;
    s.d = d;
    return s;
}
// Tokens of a row on average (packed rows' own lengths are only on the device).
inline long mean_tokens(int B, int T, bool varlen) { return varlen ? ((long)T + B - 1) / (B > 0 ? B : 1) : T; }

Plan plan_simt(int B, int T, int Hq, int Hk, int d, bool varlen);
cudaError_t launch_attention_simt(const AttentionParams &p, const Plan &s, cudaStream_t stream);
// 16-bit tensors whose addresses and strides are multiples of 16 bytes.
bool tc_takes(const AttentionParams &p);
Plan plan_tc(int B, int T, int Hq, int Hk, int d, bool varlen);
cudaError_t launch_attention_tc(const AttentionParams &p, const Plan &s, cudaStream_t stream);

}  // namespace attn

// Tensor maps of 16-bit tensors, 128-byte swizzle, 64 features to a 128-byte row (zeros past
// d).  Queries [tokens][H][d]: boxes of `heads` x `tokens` rows of 64 features.
bool encode_heads_map(CUtensorMap *m, const void *ptr, bool bf16, int d, int H, long tokens, int64_t token_stride,
                      int box_heads, int box_tokens);
// A cache's pages, as [count][slots / 8][d / 64][8 slots][64]: boxes of `rows` slots with all
// their features, 8 slots of 64 features next to each other.  `unit`: elements from one
// index of the first dimension to the next.
bool encode_pages_map(CUtensorMap *m, const void *ptr, bool bf16, int d, int slots, int64_t slot_stride, int64_t count,
                      int64_t unit, int rows);
}  // namespace gdn
