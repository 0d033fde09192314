// gdn_attention.cuh -- how the attention kernels cut their work, and join what they cut.
//
// A unit is (row b, key head hk, block of query rows): the G = Hq / Hk query heads of a key
// head and the row's tokens are flattened, rho = t G + g, so that all of them read a tile of
// keys once; a unit has up to `rows` of them, and as many tiles of `keys` keys as they see.
// All units' tiles in a row, in the order of b, hk, block, are cut into equal pieces, one a
// CTA, so that no lengths, however ragged, leave CTAs idle.  Lengths are on the device, so
// each CTA finds its piece there: a sum over the rows and a walk along the one it starts in.
// A unit that a cut goes through leaves its parts (unscaled sums, maxima, sums of weights) in
// the workspace, at most two a CTA: the end of a unit that an earlier CTA began (head) and
// the start of one that a later CTA goes on with (tail).  The join, a second kernel, adds the
// parts up in the order of the keys, so the result does not depend on timing.
#pragma once

#include "gdn_internal.cuh"
#include "tc_ptx.cuh"

namespace gdn {
namespace attn {

constexpr float kNone = -INFINITY;

// What a CTA leaves for the join.
struct alignas(16) Cut {
    int tail;          // 1: the CTA's last unit goes on in the next CTA
    int b, hk, block;  // that unit
    int head;          // 0: nothing; 1: its first unit began in an earlier CTA and ends here; 2: and goes on
    int pad[3];
};

// The cutting, with the workspace's layout: Cut [ctas], maxima and sums [ctas][2][rows][2],
// sums [ctas][2][rows][d].
struct Plan {
    int rows, keys;  // query rows of a unit, keys of a tile
    int ctas, d;
    uint8_t *ws;
    __host__ __device__ Cut *cut(int c) const { return reinterpret_cast<Cut *>(ws) + c; }
    __host__ __device__ float2 *stats(int c, int part) const {
        return reinterpret_cast<float2 *>(ws + (size_t)ctas * sizeof(Cut)) + ((size_t)c * 2 + part) * rows;
    }
    __host__ __device__ float *sums(int c, int part) const {
        return reinterpret_cast<float *>(ws + (size_t)ctas * (sizeof(Cut) + 2 * rows * sizeof(float2))) +
               ((size_t)c * 2 + part) * rows * d;
    }
    size_t bytes() const {
        return (size_t)ctas * (sizeof(Cut) + 2 * (size_t)rows * (sizeof(float2) + d * sizeof(float)));
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
    const long room = (long)p.max_pages * p.page_size;
    r.keys = len < room ? len : (int)room;
    r.first = len - r.tokens;
    return r;
}

// One unit's query rows and keys.
struct Unit {
    int rho0, rho1;  // flattened query rows
    int lo, hi;      // keys that any of them sees
    int key0, tiles; // the first tile's first key, tiles (one at least)
};

__device__ __forceinline__ Unit unit_of(const AttentionParams &p, const Plan &s, const Row &r, int G, int block) {
    Unit u;
    u.rho0 = block * s.rows;
    u.rho1 = min(u.rho0 + s.rows, r.tokens * G);
    const int t0 = u.rho0 / G, t1 = (u.rho1 - 1) / G;
    u.lo = 0;
    u.hi = r.keys;
    if (p.causal) {
        u.hi = min(u.hi, r.first + t1 + 1);
        if (p.window > 0) u.lo = max(0, r.first + t0 - p.window + 1);
    }
    u.key0 = u.lo / s.keys * s.keys;
    u.tiles = u.hi > u.lo ? (u.hi - u.key0 + s.keys - 1) / s.keys : 1;
    return u;
}

__device__ __forceinline__ int blocks_of(const Plan &s, const Row &r, int G) {
    return (r.tokens * G + s.rows - 1) / s.rows;
}

// Tiles of a row for one key head.
__device__ __forceinline__ long row_tiles(const AttentionParams &p, const Plan &s, const Row &r, int G) {
    long n = 0;
    const int blocks = blocks_of(s, r, G);
    for (int i = 0; i < blocks; ++i) n += unit_of(p, s, r, G, i).tiles;
    return n;
}

// A place in the order of all tiles, and the tiles from there to the CTA's end.
struct Place {
    int b, hk, block, tile;
    long left;
};

// Where this CTA's piece starts.  Called by all THREADS threads.
template <int THREADS>
__device__ Place find_place(const AttentionParams &p, const Plan &s, int G) {
    __shared__ long sums[THREADS / 32];
    __shared__ Place found;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int per = (p.B + THREADS - 1) / THREADS;
    const int b0 = min((int)threadIdx.x * per, p.B), b1 = min(b0 + per, p.B);
    long mine = 0;
    for (int b = b0; b < b1; ++b) mine += row_tiles(p, s, row_at(p, b), G) * p.Hk;
    long upto = mine;
    for (int o = 1; o < 32; o <<= 1) {
        const long x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    if (lane == 31) sums[warp] = upto;
    __syncthreads();
    long before = 0, total = 0;
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    before += upto - mine;
    // (no more CTAs than tiles: one without a piece never stands between a unit's parts)
    const long n = max(1l, min((long)s.ctas, total)), c = min((long)blockIdx.x, n);
    const long from = total * c / n, to = blockIdx.x < n ? total * (c + 1) / n : from;
    if (threadIdx.x == 0 && from >= to) found.left = 0;
    if (from < to && before <= from && from < before + mine) {
        long rest = from - before;
        for (int b = b0; b < b1; ++b) {
            const Row r = row_at(p, b);
            const long n = row_tiles(p, s, r, G);
            if (rest >= n * p.Hk) {
                rest -= n * p.Hk;
                continue;
            }
            found.b = b;
            found.hk = (int)(rest / n);
            rest -= found.hk * n;
            int i = 0;
            for (;; ++i) {
                const int t = unit_of(p, s, r, G, i).tiles;
                if (rest < t) break;
                rest -= t;
            }
            found.block = i;
            found.tile = (int)rest;
            found.left = to - from;
            break;
        }
    }
    __syncthreads();
    return found;
}

// The piece's units one after another.  at() gives the unit at hand, its tiles [tile, end).
struct Walk {
    Place at;
    Row row;
    Unit unit;
    int end, blocks;
    int nth;  // of this CTA's units
    __device__ __forceinline__ void load(const AttentionParams &p, const Plan &s, int G) {
        unit = unit_of(p, s, row, G, at.block);
        end = (int)min((long)unit.tiles, at.tile + at.left);
    }
    __device__ __forceinline__ bool start(const AttentionParams &p, const Plan &s, int G, const Place &from) {
        at = from;
        nth = 0;
        if (at.left <= 0) return false;
        row = row_at(p, at.b);
        blocks = blocks_of(s, row, G);
        load(p, s, G);
        return true;
    }
    __device__ __forceinline__ bool next(const AttentionParams &p, const Plan &s, int G) {
        at.left -= end - at.tile;
        if (at.left <= 0) return false;
        ++nth;
        at.tile = 0;
        if (++at.block == blocks) {
            at.block = 0;
            if (++at.hk == p.Hk) {
                at.hk = 0;
                do {
                    if (++at.b >= p.B) return false;
                    row = row_at(p, at.b);
                    blocks = blocks_of(s, row, G);
                } while (blocks == 0);
            }
        }
        load(p, s, G);
        return true;
    }
    __device__ __forceinline__ bool whole() const { return at.tile == 0 && end == unit.tiles; }
    // Which of the CTA's two parts a cut unit leaves.
    __device__ __forceinline__ int part() const { return at.tile > 0 ? 0 : 1; }
};

// What the CTA leaves for the join, written by one thread (Place `from` as found).
__device__ inline void write_cut(const AttentionParams &p, const Plan &s, int G, const Place &from) {
    Cut c{};
    Walk w;
    if (w.start(p, s, G, from)) {
        if (w.at.tile > 0) c.head = w.end == w.unit.tiles ? 1 : 2;
        do {
            if (w.at.tile == 0 && w.end < w.unit.tiles) {
                c.tail = 1;
                c.b = w.at.b;
                c.hk = w.at.hk;
                c.block = w.at.block;
            }
        } while (w.next(p, s, G));
    }
    *s.cut(blockIdx.x) = c;
}

// Joins the parts of cut units.  Grid (ctas, slices): CTA x takes the unit that CTA x of the
// attention left a tail of, a warp a query row; maxima are those of scores times log2 e.
template <typename T>
__global__ void __launch_bounds__(256) join_kernel(const AttentionParams p, const Plan s) {
    tc::grid_dependency_wait();
    const Cut c = *s.cut(blockIdx.x);
    if (!c.tail) return;
    const int G = p.Hq / p.Hk;
    const Row r = row_at(p, c.b);
    const Unit u = unit_of(p, s, r, G, c.block);
    const int lane = threadIdx.x % 32, warps = blockDim.x / 32;
    // the CTA in which the unit ends
    int last = blockIdx.x + 1;
    while (last < s.ctas - 1 && s.cut(last)->head == 2) ++last;
    const int n = u.rho1 - u.rho0, per = s.d / 32;
    for (int i = blockIdx.y * warps + threadIdx.x / 32; i < n; i += gridDim.y * warps) {
        float top = kNone;
        for (int x = blockIdx.x + lane; x <= last; x += 32)
            top = fmaxf(top, s.stats(x, x == (int)blockIdx.x)[i].x);
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const float safe = top == kNone ? 0.f : top;
        float sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int x = blockIdx.x; x <= last; ++x) {
            const int part = x == (int)blockIdx.x;
            const float2 ml = s.stats(x, part)[i];
            const float *o = s.sums(x, part) + (size_t)i * s.d + lane * per;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
            if (per == 4) {
                const float4 f = *reinterpret_cast<const float4 *>(o);
                v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
            } else if (per == 2) {
                const float2 f = *reinterpret_cast<const float2 *>(o);
                v[0] = f.x, v[1] = f.y;
            } else {
                v[0] = o[0];
            }
            const float w = exp2f(ml.x - safe);
            sum = fmaf(w, ml.y, sum);
            for (int e = 0; e < 4; ++e) acc[e] = fmaf(w, v[e], acc[e]);
        }
        const int rho = u.rho0 + i, t = rho / G;
        const long at = (r.tok0 + t) * p.Hq + c.hk * G + (rho - t * G);
        const float inv = sum > 0.f ? 1.f / sum : sum == 0.f ? 0.f : sum;  // (a NaN stays one)
        T *out = reinterpret_cast<T *>(p.out) + at * p.d + lane * per;
        for (int e = 0; e < per; ++e) st_out(out + e, acc[e] * inv);
        if (p.lse != nullptr && lane == 0) p.lse[at] = (safe + log2f(sum)) * 0.69314718055994530942f;
    }
}

// Launched behind an attention kernel, while it still runs.
cudaError_t launch_join(const AttentionParams &p, const Plan &s, cudaStream_t stream);

// Plans of the two kernels.
Plan plan_simt(int B, int T, int Hq, int Hk, int d, bool varlen);
cudaError_t launch_attention_simt(const AttentionParams &p, const Plan &s, cudaStream_t stream);
// 16-bit tensors that TMA can address, with pages of a multiple of 8 slots and up to 128
// query heads a key head.
bool tc_takes(const AttentionParams &p);
Plan plan_tc(int B, int T, int Hq, int Hk, int d, bool varlen);
cudaError_t launch_attention_tc(const AttentionParams &p, const Plan &s, cudaStream_t stream);

}  // namespace attn

// Tensor maps of 16-bit tensors, 128-byte swizzle, boxes of 64 features (zeros past d):
// [tokens][H][d] with `heads` x `tokens` boxes; [pages][heads][slots][d] with boxes of `rows`
// slots.  Strides in elements.
bool encode_heads_map(CUtensorMap *m, const void *ptr, bool bf16, int d, int H, long tokens, int64_t head_stride,
                      int64_t token_stride, int box_heads, int box_tokens);
bool encode_pages_map(CUtensorMap *m, const void *ptr, bool bf16, int d, int slots, int heads, int pages,
                      int64_t slot_stride, int64_t head_stride, int64_t page_stride, int rows);
}  // namespace gdn
