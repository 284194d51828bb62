// norm.cu -- the step between two linear layers of a decoder: the residual
// stream updated with a block's output (its own norm, gate and residual scale
// applied), the next layer's RMS norm, and, fused with them, that layer's
// rotation and quantiser (kernel K1 without the normed row in between).
//
// Per row m of K channels, all in fp32, every product and sum rounded on its
// own (no fma but in the sums of squares), e = the 16-bit or fp32 type of the stream:
//   p = y,  or  fl(fl(y * fl(w_post + off)) * ry)  with the norm after the block
//   p = fl(gate * p)                               with a gate
//   h = e(fl(H + fl(alpha * p)))                   (h = H without a block)
//   v = fl(h * fl(w + off)),  x = e(fl(v * rh))
//   rh = 1 / sqrt(fl(sum h^2 / K) + eps),  ry the same of y
// and with the quantiser
//   u = (v .* d) H_sylv per group, amax = max |u|, q = rint(fl(u * fl(7/amax)))
//   sx = fl(fl(fl(amax/7) * fl(1/sqrt(g))) * rh)   (127 in place of 7 for 8 bits)
// A symmetric per-token quantiser does not see a factor common to the row, so
// rh enters the scale only: the codes are those of the un-normed v, need no
// statistic of the row but amax, and skip the 16-bit rounding of x.
//
// Source: OffQ, Methodology 2 and 3 (the rotation), SERQ, technical summary
// section 1 (per-token symmetric 4-bit activations), DynamicPTQ, Methodology 2
// (8 bits for sensitive layers); the norm itself is the RMS norm of the Llama
// layers whose shapes the pages quote.
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "hq_device.cuh"

namespace hq {
namespace {

constexpr int NM_MAXK = 16384;

struct NormArgs {
    const void *H, *Y, *gate, *w_post, *w;
    void *Ho, *X;
    uint8_t* Xq;
    float* sx;
    const int8_t* d;
    int64_t ldh, ldy, ldg, ldho, ldx;
    int M, K, group, wt;
    float alpha, off, eps, cg;
    float2 nz;   // (-0, -0)
};

// A vector is 16 bytes of the stream: 8 values of 16 bits or 4 of fp32
template <int XT>
constexpr int vec_len = XT == HQ_F32 ? 4 : 8;

// Row m of a matrix: the same for the whole CTA, so that a vector's address is
// one uniform base and a 32-bit offset
template <int XT>
__device__ __forceinline__ const uint8_t* row_of(const void* p, int64_t m, int64_t ld) {
    return static_cast<const uint8_t*>(p) + m * ld * (XT == HQ_F32 ? 4 : 2);
}
template <int XT>
__device__ __forceinline__ uint8_t* row_of(void* p, int64_t m, int64_t ld) {
    return static_cast<uint8_t*>(p) + m * ld * (XT == HQ_F32 ? 4 : 2);
}

// The vector at byte `at` of a row, n of its values (TAIL: the row may end inside
// the vector; otherwise it is whole or absent)
template <int XT, bool TAIL>
__device__ __forceinline__ uint4 ld_vec(const uint8_t* row, uint32_t at, int n) {
    if (!TAIL || n == vec_len<XT>)
        return n > 0 ? __ldg(reinterpret_cast<const uint4*>(row + at)) : make_uint4(0u, 0u, 0u, 0u);
    uint32_t t[4] = {0u, 0u, 0u, 0u};
    if constexpr (XT == HQ_F32) {
        const float* s = reinterpret_cast<const float*>(row + at);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) t[e] = __float_as_uint(__ldg(s + e));
    } else {
        const uint16_t* s = reinterpret_cast<const uint16_t*>(row + at);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) t[e / 2] |= static_cast<uint32_t>(__ldg(s + e)) << (16 * (e & 1));
    }
    return make_uint4(t[0], t[1], t[2], t[3]);
}

template <int XT>
__device__ __forceinline__ void widen(const uint4& q, float (&v)[vec_len<XT>]) {
    const uint32_t t[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (XT == HQ_F32) {
            v[e] = __uint_as_float(t[e]);
        } else if constexpr (XT == HQ_BF16) {
            v[2 * e] = __uint_as_float(t[e] << 16);
            v[2 * e + 1] = __uint_as_float(t[e] & 0xFFFF0000u);
        } else {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&t[e]));
            v[2 * e] = f.x;
            v[2 * e + 1] = f.y;
        }
    }
}

template <int XT>
__device__ __forceinline__ uint4 narrow(const float (&v)[vec_len<XT>]) {
    uint32_t t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if constexpr (XT == HQ_F32) {
            t[e] = __float_as_uint(v[e]);
        } else if constexpr (XT == HQ_BF16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
            t[e] = *reinterpret_cast<const uint32_t*>(&b);
        } else {
            const __half2 b = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
            t[e] = *reinterpret_cast<const uint32_t*>(&b);
        }
    }
    return make_uint4(t[0], t[1], t[2], t[3]);
}

template <int XT, bool TAIL>
__device__ __forceinline__ void st_vec(uint8_t* row, uint32_t at, int n, const uint4& q) {
    if (!TAIL || n == vec_len<XT>) {
        if (n > 0) *reinterpret_cast<uint4*>(row + at) = q;
        return;
    }
    const uint32_t t[4] = {q.x, q.y, q.z, q.w};
    if constexpr (XT == HQ_F32) {
        float* s = reinterpret_cast<float*>(row + at);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (e < n) s[e] = __uint_as_float(t[e]);
    } else {
        uint16_t* s = reinterpret_cast<uint16_t*>(row + at);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) s[e] = static_cast<uint16_t>(t[e / 2] >> (16 * (e & 1)));
    }
}

// V norm weights (4 or 8) plus the offset; their type is a run-time choice (the
// branch is the same for the whole grid)
template <int V>
__device__ __forceinline__ void ld_weight(const void* w, int wt, int i, int n, float off, float (&v)[V]) {
    if (wt == HQ_F32) {
#pragma unroll
        for (int h = 0; h < V; h += 4) {
            float t[4];
            widen<HQ_F32>(ld_vec<HQ_F32, true>(static_cast<const uint8_t*>(w), 4u * (i + h), min(max(n - h, 0), 4)), t);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[h + e] = t[e];
        }
    } else {
        uint32_t t[V / 2];
        const uint16_t* s = static_cast<const uint16_t*>(w) + i;
        if (n == V) {
#pragma unroll
            for (int e = 0; e < V / 4; ++e) {
                const uint2 q = __ldg(reinterpret_cast<const uint2*>(s) + e);
                t[2 * e] = q.x;
                t[2 * e + 1] = q.y;
            }
        } else {
#pragma unroll
            for (int e = 0; e < V / 2; ++e)
                t[e] = (2 * e < n ? __ldg(s + 2 * e) : 0u) | (2 * e + 1 < n ? static_cast<uint32_t>(__ldg(s + 2 * e + 1)) << 16 : 0u);
        }
#pragma unroll
        for (int e = 0; e < V / 2; ++e) {
            const float2 f = wt == HQ_BF16 ? make_float2(__uint_as_float(t[e] << 16), __uint_as_float(t[e] & 0xFFFF0000u))
                                           : __half22float2(*reinterpret_cast<const __half2*>(&t[e]));
            v[2 * e] = f.x;
            v[2 * e + 1] = f.y;
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = __fadd_rn(v[e], off);
}

// Row-wide reductions: sums and maxima over the CTA in a fixed order, one
// barrier each.  Two buffers used in turn: a buffer is written again only after
// the next reduction's barrier, which every thread reaches after reading it.
struct RowReduce {
    float2 (*buf)[32];
    int par;
    __device__ __forceinline__ static float lanes(float s) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
        return s;
    }
    // a is not negative: its bits are ordered as it is, a NaN above infinity
    __device__ __forceinline__ static float lanes_max(float a) {
        return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(a)));
    }
    // the sum of s over the CTA; every warp adds the warps' sums for itself
    __device__ __forceinline__ float sum(float s) {
        s = lanes(s);
        if (blockDim.x > 32) {
            if ((threadIdx.x & 31) == 0) buf[par][threadIdx.x >> 5].x = s;
            __syncthreads();
            s = lanes((threadIdx.x & 31) < blockDim.x >> 5 ? buf[par][threadIdx.x & 31].x : 0.f);
            par ^= 1;
        }
        return s;
    }
    // (sum of s, max of a)
    __device__ __forceinline__ float2 sum_max(float s, float a) {
        s = lanes(s);
        a = lanes_max(a);
        if (blockDim.x > 32) {
            if ((threadIdx.x & 31) == 0) buf[par][threadIdx.x >> 5] = make_float2(s, a);
            __syncthreads();
            const float2 t = (threadIdx.x & 31) < blockDim.x >> 5 ? buf[par][threadIdx.x & 31] : make_float2(0.f, 0.f);
            s = lanes(t.x);
            a = lanes_max(t.y);
            par ^= 1;
        }
        return make_float2(s, a);
    }
};

__device__ __forceinline__ float inv_rms(float sum, int K, float eps) {
    return __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(K)), eps));
}

// ---------------------------------------------------------- without a quantiser
// A CTA walks rows m, m + grid, ...; NV vectors per thread, vector i of thread t
// at i * threads + t.  Bound by HBM (4096 x 4096 bf16 with norms on both sides and a
// gate per token: 30.3 us, 5.5 TB/s of the 6.55 of a copy; fp32 rows by their wait
// for memory, with one set of registers, and by uneven rounds: 1537 x 5003 in 28.3 us,
// 4.4 TB/s, is 5.2 rows for each of 296 CTAs, so six): the weights stay in registers
// as fp32 over the CTA's rows (KEEP) and the next row is requested before this one is
// worked on; rows whose registers do not allow both (fp32, very wide ones) have the
// weights in shared memory and request the next row at the end of this one (2048 bf16
// rows of 8192 channels 31 us, 26 at HBM's rate; of 16384 74 us, 51).  A row is in
// registers from its load to its stores.
template <int XT, int NV, bool POST, bool KEEP, bool TAIL, int MAXT>
__global__ void __launch_bounds__(MAXT, !KEEP && MAXT == 512 ? 2 : 1) k_residual_norm(const NormArgs a) {
    constexpr int V = vec_len<XT>;
    __shared__ float2 red[2][32];
    extern __shared__ __align__(16) float wsm[];   // weights (not KEEP)
    RowReduce reduce{red, 0};
    int n[NV];
    uint32_t col[NV], at[NV];   // first channel of a vector, its byte
    float wp[KEEP && POST ? NV : 1][V], wn[KEEP ? NV : 1][V];   // else of the vector at hand
    struct Row {
        uint4 h[NV], y[NV], g[NV];
    } r[KEEP ? 2 : 1];
    auto load = [&](int64_t m, Row& q) {   // the block first: its norm is the first thing needed
        if (a.Y != nullptr) {
#pragma unroll
            for (int i = 0; i < NV; ++i) q.y[i] = ld_vec<XT, TAIL>(row_of<XT>(a.Y, m, a.ldy), at[i], n[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) q.h[i] = ld_vec<XT, TAIL>(row_of<XT>(a.H, m, a.ldh), at[i], n[i]);
        if (a.Y != nullptr && a.gate != nullptr) {
#pragma unroll
            for (int i = 0; i < NV; ++i) q.g[i] = ld_vec<XT, TAIL>(row_of<XT>(a.gate, m, a.ldg), at[i], n[i]);
        }
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (i * blockDim.x + threadIdx.x) * V;
        at[i] = col[i] * (16 / V);
        n[i] = min(max(a.K - static_cast<int>(col[i]), 0), V);
    }
    load(blockIdx.x, r[0]);
    // without registers for them the weights lie in shared memory, as fp32, in slots
    // of 16 bytes that only their thread uses: w_post's, then w's, V / 4 per vector
    const uint32_t slots = NV * blockDim.x;
    auto slot = [&](int which, int i, int h) {
        return wsm + ((which * (V / 4) + h) * slots + i * blockDim.x + threadIdx.x) * 4;
    };
    auto stage_w = [&](int which, const void* w) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float f[V];
            ld_weight<V>(w, a.wt, col[i], n[i], a.off, f);
#pragma unroll
            for (int h = 0; h < V / 4; ++h)
                *reinterpret_cast<float4*>(slot(which, i, h)) = make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
        }
    };
    auto weight = [&](int which, int i, float (&f)[V]) {
#pragma unroll
        for (int h = 0; h < V / 4; ++h) {
            const float4 q = *reinterpret_cast<const float4*>(slot(which, i, h));
            f[4 * h] = q.x; f[4 * h + 1] = q.y; f[4 * h + 2] = q.z; f[4 * h + 3] = q.w;
        }
    };
    if constexpr (!KEEP) {
        if constexpr (POST) stage_w(1, a.w_post);
        if (a.w != nullptr) stage_w(0, a.w);
    }
    if constexpr (KEEP) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (POST) ld_weight<V>(a.w_post, a.wt, col[i], n[i], a.off, wp[i]);
            if (a.w != nullptr) ld_weight<V>(a.w, a.wt, col[i], n[i], a.off, wn[i]);
        }
    }
    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        Row& q = r[0];
        if constexpr (KEEP) {
            if (m + gridDim.x < a.M) load(m + gridDim.x, r[1]);
        }
        if (a.Y != nullptr) {
            float rstd = 1.f;
            if constexpr (POST) {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    float y[V];
                    widen<XT>(q.y[i], y);
#pragma unroll
                    for (int e = 0; e < V; ++e) ss = __fmaf_rn(y[e], y[e], ss);
                }
                rstd = inv_rms(reduce.sum(ss), a.K, a.eps);
            }
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float p[V], h[V];
                widen<XT>(q.y[i], p);
                widen<XT>(q.h[i], h);
                if constexpr (POST) {
                    if constexpr (!KEEP) weight(1, i, wp[0]);
#pragma unroll
                    for (int e = 0; e < V; ++e) p[e] = __fmul_rn(__fmul_rn(p[e], wp[KEEP ? i : 0][e]), rstd);
                }
                if (a.gate != nullptr) {
                    float g[V];
                    widen<XT>(q.g[i], g);
#pragma unroll
                    for (int e = 0; e < V; ++e) p[e] = __fmul_rn(g[e], p[e]);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) h[e] = __fadd_rn(h[e], __fmul_rn(a.alpha, p[e]));
                q.h[i] = narrow<XT>(h);   // what the norm reads is the stored stream
            }
        }
        if (a.Ho != nullptr) {
#pragma unroll
            for (int i = 0; i < NV; ++i) st_vec<XT, TAIL>(row_of<XT>(a.Ho, m, a.ldho), at[i], n[i], q.h[i]);
        }
        if (a.w != nullptr) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float h[V];
                widen<XT>(q.h[i], h);
#pragma unroll
                for (int e = 0; e < V; ++e) ss = __fmaf_rn(h[e], h[e], ss);
            }
            const float rstd = inv_rms(reduce.sum(ss), a.K, a.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float h[V];
                widen<XT>(q.h[i], h);
                if constexpr (!KEEP) weight(0, i, wn[0]);
#pragma unroll
                for (int e = 0; e < V; ++e) h[e] = __fmul_rn(__fmul_rn(h[e], wn[KEEP ? i : 0][e]), rstd);
                st_vec<XT, TAIL>(row_of<XT>(a.X, m, a.ldx), at[i], n[i], narrow<XT>(h));
            }
        }
        if constexpr (KEEP)
            r[0] = r[1];
        else if (m + gridDim.x < a.M)
            load(m + gridDim.x, r[0]);
    }
}

// ------------------------------------------------------------- with a quantiser
// A CTA walks rows; a warp takes 1024 consecutive channels of a row, 32 per
// thread.  The weights, with the offset added and the rotation's signs d on
// them, are staged in shared memory as fp32 once per CTA (h (w d) is exactly
// (h w) d), and the next row is requested before this one is rotated.  The
// butterfly runs in registers between shared-memory transposes of the fp32
// values (a shuffle per element and stage took 4 times the shared-memory
// instructions):
//   layout A: thread l of a warp holds channels 256 i + 8 l .. + 7, i = 0..3 (16-byte
//             loads and stores, contiguous over the warp): stages 1, 2, 4
//   layout B: channels 256 (l / 8) + l % 8 + 8 k, k = 0..31: stages 8 .. 128
//   layout D: (groups above 256) thread t of the group's g/32 threads holds
//             channels t + (g/32) q + 256 j, j = 0 .. g/256 - 1: stages 256 ..
// and back to A for the codes.  Channel c of the row is stored at c + 4 (c / 32) +
// 8 (c / 256), which makes the accesses of all layouts free of bank conflicts; the
// weights lie in slots of 16 bytes that only their lane uses.
// Measured: 2048 x 4096, group 4096, 8 bits 18.7 us (9.0 at HBM's rate); 8192 x 8192,
// group 256, 4 bits, the normed rows and a gate per channel 116 us (87), per token 125
// (107); codes only, 8192 x 4096, group 128, 4 bits 35.0 us (12.8) without a block, 43.1
// (33.3) with one.  Bound by the latency of its instructions at 16 warps per SM (128 registers):
// about 34 per value, issued at 0.5 per cycle and scheduler.  With fewer registers it
// spills and is slower; with 16 values per thread and 32 warps per SM the work per row
// and thread (reductions, divisions, addresses) weighs twice: 20.3 and 160 us.
// A and B stay within the warp; D of groups of 2048 and 4096 needs the CTA.
__host__ __device__ constexpr int nq_at(int c) { return c + 4 * (c >> 5) + 8 * (c >> 8); }
constexpr int NQ_SPAN = 1024;                 // channels of a warp
constexpr int NQ_BUF = nq_at(NQ_SPAN);        // floats for them, 1184

__device__ __forceinline__ float2 f2_add(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
// a - b, as the exact b * -1 plus a
__device__ __forceinline__ float2 f2_sub(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, n;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 n, {%6, %6};\n\t"
        "fma.rn.f32x2 z, y, n, x;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(-1.0f));
    return r;
}
__device__ __forceinline__ float2 f2_fma(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z, w;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
// a b, rounded on its own: the compiler merges a packed product, or one that it sees
// to be plus -0, with a packed sum after it, so `nz` is a -0 that it does not know
__device__ __forceinline__ float2 f2_mul(float2 a, float2 b, float2 nz) { return f2_fma(a, b, nz); }
__device__ __forceinline__ float2 f2_of(const float* v) { return make_float2(v[0], v[1]); }
__device__ __forceinline__ void f2_to(float* v, float2 a) {
    v[0] = a.x;
    v[1] = a.y;
}
// NaN if one of them is: infinities that meet in the butterfly leave NaN, and a row
// of them must not pass for one of small values
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// (a, b) -> (a + b, a - b) for the pairs of v[] whose index differs in bit S
template <int S>
__device__ __forceinline__ void stage(float (&v)[32]) {
    if constexpr (S == 1) {
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
            const float a = v[i], b = v[i + 1];
            v[i] = __fadd_rn(a, b);
            v[i + 1] = __fsub_rn(a, b);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 32; i += 2)
            if ((i & S) == 0) {
                const float2 a = make_float2(v[i], v[i + 1]), b = make_float2(v[i + S], v[i + S + 1]);
                const float2 s = f2_add(a, b), d = f2_sub(a, b);
                v[i] = s.x; v[i + 1] = s.y;
                v[i + S] = d.x; v[i + S + 1] = d.y;
            }
    }
}

// Stages 256 .. 128 J of a group of 256 J channels in layout D; `base` is the
// group's place in shared memory, t the thread's number in the group
template <int J>
__device__ __forceinline__ void stages_d(float (&v)[32], float* base, int t) {
    float* p = base + t + 4 * (t >> 5);
#pragma unroll
    for (int q = 0; q < 32 / J; ++q)
#pragma unroll
        for (int j = 0; j < J; ++j) v[q * J + j] = p[nq_at(8 * J * q) + nq_at(256) * j];   // g/32 = 8 J
    stage<1>(v);
    if constexpr (J > 2) stage<2>(v);
    if constexpr (J > 4) stage<4>(v);
    if constexpr (J > 8) stage<8>(v);
#pragma unroll
    for (int q = 0; q < 32 / J; ++q)
#pragma unroll
        for (int j = 0; j < J; ++j) p[nq_at(8 * J * q) + nq_at(256) * j] = v[q * J + j];
}

// FULL: rows of a multiple of 1024 channels, every vector is there.
// IN: the operands beside H: none, Y, or Y and the gate, whose next row is requested
// before the codes are written (at its use it cost 180 us in place of 126 at 8192 x
// 8192).  Without Y the registers allow 20 warps per SM (8192 x 4096, group 128: 35.0 us,
// 37.8 at 16; rows of more than 10 warps do not gain).
template <int XT, int BITS, bool FULL, int IN>
__global__ void __launch_bounds__(IN == 0 ? 640 : 512) k_norm_quant(const NormArgs a) {
    __shared__ float2 red[2][32];
    extern __shared__ __align__(16) float dyn[];   // weights, then the row
    // the small-M GEMM may be launched early: it waits for this grid's
    // completion before it reads the codes
    asm volatile("griddepcontrol.launch_dependents;");
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.d != nullptr && a.d[0] == -1) record_status(HQ_ERR_ARG);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col0 = warp * NQ_SPAN + lane * 8;
    const uint32_t at0 = 2 * col0;
    const int G = a.group;
    RowReduce reduce{red, 0};
    float* row = dyn + (blockDim.x >> 5) * NQ_SPAN;
    float* buf = row + warp * NQ_BUF;
    float* wrow = dyn + warp * NQ_SPAN + 4 * lane;   // + 256 i + 128 h: weights of half h of vector i
    bool on[4];   // K is a multiple of 32: vectors are whole or absent
#pragma unroll
    for (int i = 0; i < 4; ++i) on[i] = FULL || col0 + 256 * i < a.K;

    struct Row {
        uint4 h[4], y[4];
    } r;
    auto load = [&](int64_t m, Row& q) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q.h[i] = ld_vec<XT, false>(row_of<XT>(a.H, m, a.ldh), at0 + 512 * i, on[i]);
        if constexpr (IN > 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                q.y[i] = ld_vec<XT, false>(row_of<XT>(a.Y, m, a.ldy), at0 + 512 * i, on[i]);
        }
    };
    load(blockIdx.x, r);
    uint4 gv[4];
    if constexpr (IN > 1) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            gv[i] = ld_vec<XT, false>(row_of<XT>(a.gate, blockIdx.x, a.ldg), at0 + 512 * i, on[i]);
    }
    // weights of this lane's channels (each lane reads back what it wrote), and the
    // signs of d: those of pair 4 i + e / 2 in bits 15 and 31 less the pair's number
    uint32_t neg = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (on[i]) {
            float w[8];
            ld_weight<8>(a.w, a.wt, col0 + 256 * i, 8, a.off, w);
            if (a.d != nullptr) {
                const int8_t* d = a.d + ((col0 + 256 * i) & (G - 1));
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (d[e] == -1) {
                        neg |= 1u << (((e & 1) ? 31 : 15) - 4 * i - e / 2);
                        w[e] = -w[e];
                    }
            }
            *reinterpret_cast<float4*>(wrow + 256 * i) = make_float4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<float4*>(wrow + 256 * i + 128) = make_float4(w[4], w[5], w[6], w[7]);
        }
    }
    const int ia = 8 * lane + 4 * (lane >> 2);               // layout A: nq_at(8 l); + nq_at(256) i
    const int ib = nq_at(256) * (lane >> 3) + (lane & 7);    // layout B: + nq_at(8 k)
    float* gbase = nullptr;                                  // layout D: the group and the thread's number in it
    int gt = 0;
    if (G > 256) {
        const int tg = G / 32;
        gt = threadIdx.x & (tg - 1);
        gbase = row + (threadIdx.x / tg) * ((G >> 8) * nq_at(256));
    }

    for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
        // ---- the residual stream after the block, v = h (w + off) d
        float v[32];
        float2 ss2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float h[8];
            widen<XT>(r.h[i], h);
            if constexpr (IN > 0) {
                float p[8];
                widen<XT>(r.y[i], p);
                if constexpr (IN > 1) {
                    float g[8];
                    widen<XT>(gv[i], g);
#pragma unroll
                    for (int e = 0; e < 8; e += 2) f2_to(p + e, f2_mul(f2_of(g + e), f2_of(p + e), a.nz));
                }
#pragma unroll
                for (int e = 0; e < 8; e += 2)
                    f2_to(h + e, f2_add(f2_of(h + e), f2_mul(make_float2(a.alpha, a.alpha), f2_of(p + e), a.nz)));
                r.h[i] = narrow<XT>(h);
                widen<XT>(r.h[i], h);   // what the norm reads is the stored stream
            }
            if (a.Ho != nullptr) st_vec<XT, false>(row_of<XT>(a.Ho, m, a.ldho), at0 + 512 * i, on[i], r.h[i]);
            if (on[i]) {
                const float4 w0 = *reinterpret_cast<const float4*>(wrow + 256 * i);
                const float4 w1 = *reinterpret_cast<const float4*>(wrow + 256 * i + 128);
                const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    ss2 = f2_fma(f2_of(h + e), f2_of(h + e), ss2);
                    f2_to(v + 8 * i + e, f2_mul(f2_of(h + e), f2_of(w + e), a.nz));
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * i + e] = 0.f;
            }
        }
        const float ss = __fadd_rn(ss2.x, ss2.y);
        if (m + gridDim.x < a.M) load(m + gridDim.x, r);   // arrives while this row is rotated
        if (a.X != nullptr) {
            const float rstd = inv_rms(reduce.sum(ss), a.K, a.eps);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (on[i]) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; e += 2) f2_to(x + e, f2_mul(f2_of(v + 8 * i + e), make_float2(rstd, rstd), a.nz));
                    uint4 q = narrow<XT>(x);   // without the signs
                    q.x ^= (neg << (4 * i)) & 0x80008000u;
                    q.y ^= (neg << (4 * i + 1)) & 0x80008000u;
                    q.z ^= (neg << (4 * i + 2)) & 0x80008000u;
                    q.w ^= (neg << (4 * i + 3)) & 0x80008000u;
                    st_vec<XT, false>(row_of<XT>(a.X, m, a.ldx), at0 + 512 * i, 1, q);
                }
        }
        // ---- butterfly, stages in ascending order
        stage<1>(v);
        stage<2>(v);
        stage<4>(v);
        float amax[4] = {0.f, 0.f, 0.f, 0.f};
        if (G > 8) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 8; e += 4)
                    *reinterpret_cast<float4*>(buf + ia + nq_at(256) * i + e) =
                        make_float4(v[8 * i + e], v[8 * i + e + 1], v[8 * i + e + 2], v[8 * i + e + 3]);
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = buf[ib + nq_at(8 * k)];
            stage<1>(v);
            if (G > 16) stage<2>(v);
            if (G > 32) stage<4>(v);
            if (G > 64) stage<8>(v);
            if (G > 128) stage<16>(v);
            // each thread writes where it read
#pragma unroll
            for (int k = 0; k < 32; ++k) buf[ib + nq_at(8 * k)] = v[k];
            if (G > 256) {
                if (G > NQ_SPAN)
                    __syncthreads();
                else
                    __syncwarp();
                if (G == 512)
                    stages_d<2>(v, gbase, gt);
                else if (G == 1024)
                    stages_d<4>(v, gbase, gt);
                else if (G == 2048)
                    stages_d<8>(v, gbase, gt);
                else
                    stages_d<16>(v, gbase, gt);
            }
        }
#pragma unroll
        for (int k = 0; k < 32; k += 2) amax[(k >> 1) & 3] = max3_abs(amax[(k >> 1) & 3], v[k], v[k + 1]);
        // ---- row scale; back to layout A
        const float2 t = reduce.sum_max(ss, max3_abs(max3_abs(amax[0], amax[1], amax[2]), amax[3], 0.f));
        if (G > 8) {
            __syncwarp();   // one warp per row: the reduction has no barrier
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 8; e += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(buf + ia + nq_at(256) * i + e);
                    v[8 * i + e] = f.x; v[8 * i + e + 1] = f.y; v[8 * i + e + 2] = f.z; v[8 * i + e + 3] = f.w;
                }
        }
        if (m + gridDim.x < a.M) {
        if constexpr (IN > 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                gv[i] = ld_vec<XT, false>(row_of<XT>(a.gate, m + gridDim.x, a.ldg), at0 + 512 * i, on[i]);
        }
        }
        constexpr float LEVELS = BITS == 8 ? 127.0f : 7.0f;
        float inv = __fdiv_rn(LEVELS, t.y);
        if (inv == INFINITY) {   // amax is 0 or tiny
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = sign_of(v[k]);
            inv = LEVELS;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!on[i]) continue;
            uint8_t* qrow = a.Xq + m * (BITS == 8 ? a.K : a.K / 2);
            const uint32_t at = BITS == 8 ? col0 + 256 * i : (col0 + 256 * i) / 2;
            // fl(u * inv) is at most LEVELS (1 + 2^-23): adding 1.5 * 2^23 (+ 8 for
            // unsigned nibbles) rounds it to an integer, ties to even, whose bits end
            // the sum.  The product is rounded on its own.
            constexpr float MAGIC = BITS == 8 ? 12582912.0f : 12582920.0f;
            uint32_t c[8];
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 s = f2_add(f2_mul(f2_of(v + 8 * i + e), make_float2(inv, inv), a.nz), make_float2(MAGIC, MAGIC));
                c[e] = __float_as_uint(s.x);
                c[e + 1] = __float_as_uint(s.y);
            }
            if constexpr (BITS == 8) {
                const uint32_t lo = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
                const uint32_t hi = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
                *reinterpret_cast<uint2*>(qrow + at) = make_uint2(lo, hi);
            } else {
                // the low byte of c + 16 c' is two nibbles q + 8; flipping their top bits
                // makes them two's complement
                uint32_t b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) b[e] = c[2 * e] + (c[2 * e + 1] << 4);
                *reinterpret_cast<uint32_t*>(qrow + at) =
                    __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410) ^ 0x88888888u;
            }
        }
        // a NaN or infinity among the rotated values makes the scale NaN: of an infinite
        // amax and rstd = 0 nothing else would remain of it
        if (threadIdx.x == 0) {
            const float rstd = inv_rms(t.x, a.K, a.eps);
            const float sx = t.y == 0.f ? 0.f : __fmul_rn(__fmul_rn(__fdiv_rn(t.y, LEVELS), a.cg), rstd);
            a.sx[m] = t.y < INFINITY ? sx : NAN;
        }
    }
}

bool nm_al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool nm_type(int t) { return t == HQ_F16 || t == HQ_BF16 || t == HQ_F32; }

// One CTA per row, or as many as the current device holds at once; 0 on an error
template <class Kern>
unsigned grid_for(Kern kern, int threads, int smem, int64_t M) {
    if (M <= 128) return static_cast<unsigned>(M);   // the least that a device of this kind holds: no need to ask
    int dev = 0, per_sm = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, smem) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || per_sm < 1)
        return 0;
    const int64_t n = static_cast<int64_t>(per_sm) * sms;
    return static_cast<unsigned>(n < M ? n : M);
}

template <int XT>
hq_status launch_norm(const NormArgs& a, cudaStream_t st) {
    // vectors per thread in blocks of up to 512 threads, and in larger ones
    constexpr int V = vec_len<XT>, NV = XT == HQ_F32 ? 3 : 2, NW = XT == HQ_F32 ? 4 : 2;
    const int vecs = (a.K + V - 1) / V;
    const bool small = vecs <= 512 * NV;
    const int nv = small ? NV : NW, threads = ((vecs + nv - 1) / nv + 31) / 32 * 32;   // at most 1024
    // up to 512 threads have 128 registers each, enough to keep the weights
    constexpr bool KEEP = XT != HQ_F32;
    const bool tail = a.K % V != 0;
    auto pick = [&](auto post) {
        constexpr bool P = decltype(post)::value;
        return small ? tail ? k_residual_norm<XT, NV, P, KEEP, true, 512> : k_residual_norm<XT, NV, P, KEEP, false, 512>
               : tail ? k_residual_norm<XT, NW, P, false, true, 1024>
                      : k_residual_norm<XT, NW, P, false, false, 1024>;
    };
    auto kern = a.w_post != nullptr ? pick(std::true_type{}) : pick(std::false_type{});
    const int smem = KEEP && small ? 0 : (a.w_post != nullptr ? 2 : 1) * nv * threads * V * 4;
    static SmemOptIn opt_in[8];
    if (!allow_smem(opt_in[(small ? 1 : 0) + (tail ? 2 : 0) + (a.w_post != nullptr ? 4 : 0)], kern, smem)) return HQ_ERR_CUDA;
    const unsigned grid = grid_for(kern, threads, smem, a.M);
    if (grid == 0) return HQ_ERR_CUDA;
    kern<<<grid, threads, smem, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

template <int XT, int BITS>
hq_status launch_norm_quant(const NormArgs& a, cudaStream_t st) {
    const int warps = (a.K + NQ_SPAN - 1) / NQ_SPAN;
    const int smem = warps * (NQ_BUF + NQ_SPAN) * static_cast<int>(sizeof(float));
    const bool full = a.K % NQ_SPAN == 0;
    const int in = a.Y == nullptr ? 0 : a.gate == nullptr ? 1 : 2;
    auto pick = [&](auto f) {
        constexpr bool F = decltype(f)::value;
        return in == 0 ? k_norm_quant<XT, BITS, F, 0> : in == 1 ? k_norm_quant<XT, BITS, F, 1> : k_norm_quant<XT, BITS, F, 2>;
    };
    auto kern = full ? pick(std::true_type{}) : pick(std::false_type{});
    static SmemOptIn opt_in[6];
    if (!allow_smem(opt_in[(full ? 3 : 0) + in], kern, smem)) return HQ_ERR_CUDA;
    const unsigned grid = grid_for(kern, 32 * warps, smem, a.M);
    if (grid == 0) return HQ_ERR_CUDA;
    kern<<<grid, 32 * warps, smem, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

// Checks shared by the two entry points; the strides are in elements.
hq_status nm_check(const NormArgs& a, int64_t M, int64_t K, int xt) {
    if (M < 0 || K <= 0 || !nm_type(xt) || !nm_type(a.wt) || !(a.eps >= 0.f)) return HQ_ERR_ARG;
    if (M == 0) return HQ_OK;
    if (a.ldh < K || (a.Y && a.ldy < K) || (a.Ho && a.ldho < K) || (a.X && a.ldx < K)) return HQ_ERR_ARG;
    if (a.gate && a.ldg != 0 && a.ldg < K) return HQ_ERR_ARG;
    if (!a.Y && (a.gate || a.w_post)) return HQ_ERR_ARG;
    // in place means the same place: rows of another stride would overlap
    if (a.Ho && a.Ho == a.X) return HQ_ERR_ARG;
    if ((a.Ho == a.H && a.Ho && a.ldho != a.ldh) || (a.Ho == a.Y && a.Y && a.ldho != a.ldy) ||
        (a.X == a.H && a.X && a.ldx != a.ldh) || (a.X == a.Y && a.Y && a.ldx != a.ldy))
        return HQ_ERR_ARG;
    if (M > INT32_MAX || K > NM_MAXK) return HQ_ERR_UNSUPPORTED;
    if (!a.H) return HQ_ERR_ARG;
    const int64_t es = xt == HQ_F32 ? 4 : 2;
    for (const void* p : {a.H, a.Y, a.gate, a.w_post, a.w, static_cast<const void*>(a.Ho), static_cast<const void*>(a.X)})
        if (!nm_al16(p)) return HQ_ERR_ALIGN;
    for (int64_t ld : {a.ldh, a.Y ? a.ldy : 0, a.gate ? a.ldg : 0, a.Ho ? a.ldho : 0, a.X ? a.ldx : 0})
        if (ld * es % 16 != 0) return HQ_ERR_ALIGN;
    return HQ_OK;
}

}  // namespace
}  // namespace hq

using namespace hq;

extern "C" hq_status hq_residual_norm(const void* H, int64_t ld_h, const void* Y, int64_t ld_y, hq_dtype xt, int64_t M,
                                      int64_t K, const void* w_post, const void* gate, int64_t ld_gate, float alpha,
                                      const void* w, hq_dtype wt, float w_offset, float eps, void* H_out,
                                      int64_t ld_ho, void* X, int64_t ld_x, void* stream) {
    NormArgs a = {};
    a.H = H; a.Y = Y; a.gate = gate; a.w_post = w_post; a.w = w; a.Ho = H_out; a.X = X;
    a.ldh = ld_h; a.ldy = ld_y; a.ldg = ld_gate; a.ldho = ld_ho; a.ldx = ld_x;
    a.wt = wt; a.alpha = alpha; a.off = w_offset; a.eps = eps;
    if (M > 0 && (w == nullptr) != (X == nullptr)) return HQ_ERR_ARG;
    if (M > 0 && !X && !H_out) return HQ_ERR_ARG;
    const hq_status s = nm_check(a, M, K, xt);
    if (s != HQ_OK || M == 0) return s;
    a.M = static_cast<int>(M);
    a.K = static_cast<int>(K);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (xt == HQ_F16) return launch_norm<HQ_F16>(a, st);
    if (xt == HQ_BF16) return launch_norm<HQ_BF16>(a, st);
    return launch_norm<HQ_F32>(a, st);
}

extern "C" hq_status hq_norm_rotate_quant(const void* H, int64_t ld_h, const void* Y, int64_t ld_y, hq_dtype xt,
                                          int64_t M, int64_t K, const void* gate, int64_t ld_gate, float alpha,
                                          const void* w, hq_dtype wt, float w_offset, float eps, int32_t group,
                                          const int8_t* H_signs, int32_t bits, void* H_out, int64_t ld_ho, void* X,
                                          int64_t ld_x, void* Xq, float* sx, void* stream) {
    NormArgs a = {};
    a.H = H; a.Y = Y; a.gate = gate; a.w = w; a.Ho = H_out; a.X = X;
    a.Xq = static_cast<uint8_t*>(Xq); a.sx = sx; a.d = H_signs;
    a.ldh = ld_h; a.ldy = ld_y; a.ldg = ld_gate; a.ldho = ld_ho; a.ldx = ld_x;
    a.wt = wt; a.alpha = alpha; a.off = w_offset; a.eps = eps;
    if (group < 8 || group > 4096 || (group & (group - 1)) != 0 || (bits != 4 && bits != 8)) return HQ_ERR_ARG;
    if (K % group != 0 || K % 32 != 0) return HQ_ERR_ARG;
    if (xt == HQ_F32) return HQ_ERR_UNSUPPORTED;
    const hq_status s = nm_check(a, M, K, xt);
    if (s != HQ_OK || M == 0) return s;
    if (!w || !Xq || !sx) return HQ_ERR_ARG;
    if (!nm_al16(Xq)) return HQ_ERR_ALIGN;
    a.M = static_cast<int>(M);
    a.K = static_cast<int>(K);
    a.group = group;
    a.nz = make_float2(-0.0f, -0.0f);
    a.cg = static_cast<float>(1.0 / __builtin_sqrt(static_cast<double>(group)));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (xt == HQ_F16) return bits == 8 ? launch_norm_quant<HQ_F16, 8>(a, st) : launch_norm_quant<HQ_F16, 4>(a, st);
    return bits == 8 ? launch_norm_quant<HQ_BF16, 8>(a, st) : launch_norm_quant<HQ_BF16, 4>(a, st);
}
