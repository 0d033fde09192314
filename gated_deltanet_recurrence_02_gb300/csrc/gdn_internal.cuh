// gdn_internal.cuh -- parameter blocks, launchers and small device helpers
// shared by the libgdn kernels.  Not part of the public ABI (include/gdn.h).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/gdn.h"

namespace gdn {

// Every parameter block carries `err`: the device address of the library's
// error word (GDN_DEVERR_* bits), resolved by the host layer per device, and
// `wait_ns`: the limit of waits on another warp's work (kDefaultWaitNs unless
// a test lowered it with gdn_set_wait_limit_ns).  Waits for a CTA's own copies
// in flight, before it exits, always use kDefaultWaitNs.
constexpr uint64_t kDefaultWaitNs = 1000000000ull;

// ---------------------------------------------------------------- params --

struct RecurrentParams {
    const void *q, *k, *v, *alpha, *beta;
    const int32_t *cu_seqlens;
    const float *s0;
    const int32_t *s0_idx;
    int n_s0;
    float *s_final;
    void *out;
    int B, T, Hk, Hv, dk, dv;
    float scale;
    int dt_qkv, dt_gate;
    int conv;  // GDN_QK_L2NORM | GDN_ALPHA_LOG | GDN_BETA_LOGIT | GDN_ALPHA_PER_HEAD bits
    bool linear;  // linear attention: no beta, delta = v
    int capacity;
    const int32_t *capture_count;
    const int32_t *active;
    float *su;
    // Fused replay + verify: before the tokens, replay the first
    // clamp(rp_accepted[b], 0, rp_capacity) slots of rp_su onto the state and
    // write the result to s_commit.  rp_capacity == 0 and s_commit == nullptr
    // for the plain recurrent path.
    const float *rp_su;
    int rp_capacity;
    const int32_t *rp_accepted;
    float *s_commit;
    uint64_t wait_ns;
    uint32_t *err;
};

struct ReplayParams {
    const float *s_in;
    float *s_out;
    const float *su;
    int capacity;
    const int32_t *accepted;
    int B, Hk, Hv, dk, dv;
    uint64_t wait_ns;
    uint32_t *err;
};

struct PrefillParams {
    const void *q, *k, *v, *alpha, *beta;
    const int32_t *cu_seqlens;
    const float *s0;
    const int32_t *s0_idx;
    int n_s0;
    float *s_final;
    void *out;
    int B, T, Hk, Hv, dk, dv, chunk;
    float scale;
    int dt_qkv, dt_gate;
    int conv;  // GDN_QK_L2NORM | GDN_ALPHA_LOG | GDN_BETA_LOGIT bits
    void *ws;
    size_t ws_bytes;
    // Chunk-boundary checkpoints (nullptr: none): slot j of row b receives the
    // state after (j + 1) * ckpt_every chunks, for j < ckpt_cap, when that
    // boundary lies inside the row.  Layout [B, ckpt_cap, Hv, dv, dk].
    float *ckpt;
    int ckpt_cap, ckpt_every;
    // Compact capture as on the recurrent path (capacity 0: none): tokens
    // t < n_b of row b write decay, shared key and delta into slot t; while
    // inactive the whole [B, capacity, slot] buffer is zeroed instead.
    int capacity;
    const int32_t *capture_count;
    const int32_t *active;
    float *su;
    // Packed rows on the tensor-core path: the first global chunk index of
    // every row (B + 1 entries), written into the head of the workspace by a
    // prologue kernel; nullptr for uniform rows.
    const int32_t *chunk_table;
    uint64_t wait_ns;
    uint32_t *err;
};

// Rows are (token n, head h): element i of row (n, h) of x is x[n * xs + h * d + i].
struct GatedNormParams {
    const void *x, *z, *w;
    void *out;
    int64_t N;
    int H, d;
    int64_t xs, zs, os;
    float eps;
    int gate;  // GDN_GATE_* | GDN_GATE_FIRST | GDN_NORM_UNIT_OFFSET
    int dt_x, dt_w;
};

struct ResidualNormParams {
    const void *y, *x, *z, *w_post, *w_pre;
    void *x_out, *out;
    int64_t N;
    int D;
    int64_t ys, zs;
    float scale, eps;
    int flags;  // GDN_GATE_* | GDN_NORM_UNIT_OFFSET
    int dt_x, dt_res, dt_w;
    uint64_t wait_ns;
    uint32_t *err;
};

struct AcceptParams {
    const void *p, *q;
    const int32_t *drafts;
    const float *u;
    const int32_t *count;
    int32_t *tokens, *emitted;
    int B, K, V;
    int64_t ps, qs;
    int dt;
    uint32_t *err;
};

// Rotation of queries (or any heads: gdn_rotary has only these), and keys and values on
// their way into a paged cache.  Element (n, h, i) of q is q[n * qs + h * d + i], of k and
// v with ks and vs; of a page's slot page * page_stride + slot * slot_stride + h *
// head_stride + i.
struct RotaryParams {
    const void *q, *k, *v;
    void *q_out, *k_pages, *v_pages;
    int64_t N, qs, ks, vs, os;
    int64_t page_stride, slot_stride, head_stride;
    const int32_t *pos, *axes;  // [A, N] (nullptr: cache positions), [R / 2] or nullptr
    const float *inv_freq;
    const int32_t *page_table, *kv_lens, *cu_seqlens;
    int B, T, Hq, Hk, d, R, A, page_size, num_pages, max_pages;
    int flags, dt;  // GDN_ROTARY_*
    uint32_t *err;
};

// Attention over a paged cache (gdn_paged_attention).
struct AttentionParams {
    const void *q, *k_pages, *v_pages;
    const int32_t *page_table, *kv_lens, *cu_seqlens;
    void *out;
    float *lse;
    int B, T, Hq, Hk, d, page_size, num_pages, max_pages;
    int64_t qs, page_stride, slot_stride, head_stride;
    float scale;
    int window;
    bool causal;
    int dt;
    void *ws;
    uint64_t wait_ns;
    uint32_t *err;
};

constexpr int kRotaryMaxHeads = 16384, kRotaryMaxWidth = 1024;
constexpr int kNormMaxWidth = 16384;
constexpr int kAcceptMaxVocab = 1 << 22;   // sums of 2^40 units a token stay below 2^62
constexpr int kAcceptMaxDrafts = 1024;

// Captured tokens of row b (row length len): n_b = clamp(count, 0, min(capacity, len)),
// 0 when capture is off or inactive.
__device__ __forceinline__ int prefill_ncap(const PrefillParams &p, int b, int len) {
    if (p.capacity <= 0 || (p.active != nullptr && *p.active == 0)) return 0;
    const int c = p.capture_count[b];
    const int lim = p.capacity < len ? p.capacity : len;
    return c < 0 ? 0 : (c > lim ? lim : c);
}

// Inactive capture: CTA `cta` of `ncta` zeroes its share of the whole buffer.
__device__ __forceinline__ void prefill_capture_clear(const PrefillParams &p, long slot, long cta, long ncta,
                                                      int tid, int nthreads) {
    if (p.capacity <= 0 || p.active == nullptr || *p.active != 0) return;
    const long total = (long)p.B * p.capacity * slot;
    const long per = (total + ncta - 1) / ncta;
    const long e0 = cta * per;
    const long e1 = (e0 + per < total) ? e0 + per : total;
    for (long e = e0 + tid; e < e1; e += nthreads) p.su[e] = 0.0f;
}

// Checkpoint slot written at the end of chunk cc (0-based) of a row of len
// tokens, or -1.
__host__ __device__ __forceinline__ int ckpt_slot(const PrefillParams &p, int cc, int len) {
    if (p.ckpt == nullptr) return -1;
    const int done = cc + 1;
    if (done % p.ckpt_every != 0 || (long)done * p.chunk > len) return -1;
    const int j = done / p.ckpt_every - 1;
    return j < p.ckpt_cap ? j : -1;
}

// Launchers: enqueue on `stream`, return cudaGetLastError().
cudaError_t launch_recurrent(const RecurrentParams &p, cudaStream_t stream);
cudaError_t launch_replay(const ReplayParams &p, cudaStream_t stream);
cudaError_t launch_prefill_simt(const PrefillParams &p, cudaStream_t stream);
bool prefill_simt_supported(int dk, int dv, int chunk);
cudaError_t launch_prefill_tc(const PrefillParams &p, cudaStream_t stream);
bool prefill_tc_supported(int dk, int dv, int chunk, int dt_qkv);
size_t prefill_tc_workspace_bytes(int B, int T, int Hk, int Hv, bool varlen);

// Linear attention, chunked form on the 5th-generation tensor cores (16-bit
// inputs).  PrefillParams without beta, chunk, checkpoints and capture.
cudaError_t launch_linear_tc(const PrefillParams &p, cudaStream_t stream);
bool linear_tc_supported(int dk, int dv, int dt_qkv);
size_t linear_tc_workspace_bytes(int B, int T, int Hv, int dk, int dv, bool varlen);
// The same for fp32 inputs, on the CUDA cores.
cudaError_t launch_linear_f32(const PrefillParams &p, cudaStream_t stream);
size_t linear_f32_workspace_bytes(int B, int T, int Hv, int dk, int dv, bool varlen);
cudaError_t launch_gated_norm(const GatedNormParams &p, cudaStream_t stream);
cudaError_t launch_residual_norm(const ResidualNormParams &p, cudaStream_t stream);
cudaError_t launch_accept(const AcceptParams &p, cudaStream_t stream);
cudaError_t launch_rotary(const RotaryParams &p, cudaStream_t stream);
cudaError_t launch_attention(const AttentionParams &p, cudaStream_t stream);
size_t attention_workspace_bytes(int B, int T, int Hq, int Hk, int d, int dt, bool varlen);

// Raises kernel Kern's dynamic shared-memory limit to `bytes`, once per device
// (function attributes belong to the device's context): later calls make no
// CUDA call, so launches captured into a CUDA graph carry none.
template <auto Kern>
inline cudaError_t set_smem_once(int bytes) {
    static std::atomic<uint64_t> done{0};  // one bit per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = (dev >= 0 && dev < 64) ? (1ull << dev) : 0ull;
    if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
    e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && bit != 0) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

// Multiprocessor count of the current device, cached per device (0..63) so
// that calls after the first make no CUDA call.
inline int sm_count_of_current_device() {
    static std::atomic<int> cache[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    if (dev >= 0 && dev < 64) {
        const int c = cache[dev].load(std::memory_order_relaxed);
        if (c > 0) return c;
    }
    int v = 0;
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) return 1;
    if (dev >= 0 && dev < 64) cache[dev].store(v, std::memory_order_relaxed);
    return v;
}

// ------------------------------------------------------------- helpers --

// n / d for any 32-bit n by a multiplication: T. Granlund and P. Montgomery, "Division by
// invariant integers using multiplication" (1994), figure 4.1.
struct Divisor {
    uint32_t m, s1, s2, d;
    explicit Divisor(uint32_t d_) : d(d_) {
        uint32_t l = 0;
        while (l < 32 && (1ull << l) < d) ++l;
        m = (uint32_t)((((1ull << l) - d) << 32) / d + 1);
        s1 = l < 1 ? l : 1;
        s2 = l < 1 ? 0 : l - 1;
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const {
        const uint32_t t = __umulhi(m, n);
        return (t + ((n - t) >> s1)) >> s2;
    }
    __device__ __forceinline__ uint32_t rest(uint32_t n) const { return n - div(n) * d; }
};

__device__ __forceinline__ float ld_f(const float *p) { return *p; }
__device__ __forceinline__ float ld_f(const __half *p) { return __half2float(*p); }
__device__ __forceinline__ float ld_f(const __nv_bfloat16 *p) { return __bfloat162float(*p); }

// Four consecutive elements widened to fp32 (p 16-byte aligned for float,
// 8-byte aligned for the 16-bit types).
__device__ __forceinline__ float4 ld4(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ float4 ld4(const __half *p) {
    uint2 u = *reinterpret_cast<const uint2 *>(p);
    float2 a = __half22float2(*reinterpret_cast<__half2 *>(&u.x));
    float2 b = __half22float2(*reinterpret_cast<__half2 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float4 ld4(const __nv_bfloat16 *p) {
    uint2 u = *reinterpret_cast<const uint2 *>(p);
    float2 a = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&u.x));
    float2 b = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}

// Eight consecutive fp32 values as one 32-byte access (p 32-byte aligned).  Where
// lanes are rows apart, 16-byte accesses use half of each sector that they move,
// and meet its other half only if L1 still has it.
__device__ __forceinline__ void ld8_wide(const float *p, float2 &a, float2 &b, float2 &c, float2 &d) {
    asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(a.x), "=f"(a.y), "=f"(b.x), "=f"(b.y), "=f"(c.x), "=f"(c.y), "=f"(d.x), "=f"(d.y)
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void st8_wide(float *p, float2 a, float2 b, float2 c, float2 d) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(a.x), "f"(a.y), "f"(b.x),
                 "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y)
                 : "memory");
}

// Store fp32 as the output type, round-to-nearest-even.
__device__ __forceinline__ void st_out(float *p, float x) { *p = x; }
__device__ __forceinline__ void st_out(__half *p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void st_out(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// The same, as a volatile read-only load: it is issued where it is written,
// so that a load meant to run ahead of its use is not moved next to it.
__device__ __forceinline__ float ld_gate_early(const void *p, long idx, int dt) {
    if (dt == GDN_F32) {
        float x;
        asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(x) : "l"(reinterpret_cast<const float *>(p) + idx));
        return x;
    }
    unsigned short u;
    asm volatile("ld.global.nc.b16 %0, [%1];" : "=h"(u) : "l"(reinterpret_cast<const unsigned short *>(p) + idx));
    if (dt == GDN_F16) return __half2float(__ushort_as_half(u));
    return __bfloat162float(__ushort_as_bfloat16(u));
}

// Gate value (alpha / beta) of runtime dtype `dt` at element `idx`.
__device__ __forceinline__ float ld_gate(const void *p, long idx, int dt) {
    if (dt == GDN_F32) return reinterpret_cast<const float *>(p)[idx];
    if (dt == GDN_F16) return __half2float(reinterpret_cast<const __half *>(p)[idx]);
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[idx]);
}

// Token range [tok0, tok0 + len) of row b.  With cu_seqlens, T is the
// total token count the host validated the buffers for, and the bounds read
// from the device are clamped to [0, T] so that no access leaves the inputs.
__device__ __forceinline__ void row_range(const int32_t *cu, int b, int T,
                                          long &tok0, int &len) {
    if (cu == nullptr) {
        tok0 = (long)b * T;
        len = T;
        return;
    }
    const long total = T;
    long a = cu[b], e = cu[b + 1];
    a = a < 0 ? 0 : (a > total ? total : a);
    e = e < a ? a : (e > total ? total : e);
    tok0 = a;
    len = (int)(e - a);
}

// Initial-state matrix of (row b, head h) or nullptr for zeros.
__device__ __forceinline__ const float *initial_state_ptr(const float *s0, const int32_t *idx,
                                                          int n_s0, int b, int h, int Hv,
                                                          int dv, int dk, uint32_t *err) {
    if (s0 == nullptr) return nullptr;
    long src = b;
    if (idx != nullptr) {
        src = idx[b];
        if (src < 0 || src >= n_s0) {
            atomicOr(err, (uint32_t)GDN_DEVERR_BAD_INDEX);
            return nullptr;
        }
    }
    return s0 + ((src * Hv + h) * (long)dv) * dk;
}

// Input conventions: the decay and the write strength from the stored gates,
// and the L2-normalisation factor of a q or k vector with squared norm ss.
__device__ __forceinline__ float conv_alpha(float x, int conv) {
    return (conv & GDN_ALPHA_LOG) ? expf(x) : x;
}
__device__ __forceinline__ float conv_log_alpha(float x, int conv) {
    return (conv & GDN_ALPHA_LOG) ? x : logf(x);
}
__device__ __forceinline__ float conv_beta(float x, int conv) {
    return (conv & GDN_BETA_LOGIT) ? 1.0f / (1.0f + expf(-x)) : x;
}
__device__ __forceinline__ float l2norm_factor(float ss) { return rsqrtf(ss + 1e-6f); }

template <int W>
__device__ __forceinline__ float group_sum(float x) {
    // butterfly sum over aligned groups of W lanes (W a power of two <= 32)
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

}  // namespace gdn
