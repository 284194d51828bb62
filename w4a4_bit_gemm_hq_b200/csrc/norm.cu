// norm.cu -- the step between two linear layers of a decoder: the residual
// stream updated with a block's output (its own norm, gate and residual scale
// applied), the next layer's RMS norm, and, fused with them, that layer's
// rotation and quantiser (kernel K1 without the normed row in between).
//
// Per row m of K channels, all in fp32, every product and sum rounded on its
// own (no fma), e = the 16-bit or fp32 type of the stream:
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
};

// A vector is 16 bytes of the stream: 8 values of 16 bits or 4 of fp32
template <int XT>
constexpr int vec_len = XT == HQ_F32 ? 4 : 8;

// n < vec_len values: the row ends inside the vector
template <int XT>
__device__ __forceinline__ uint4 ld_vec(const void* p, int64_t i, int n) {
    if constexpr (XT == HQ_F32) {
        const float* s = static_cast<const float*>(p) + i;
        if (n == 4) return __ldg(reinterpret_cast<const uint4*>(s));
        return make_uint4(n > 0 ? __float_as_uint(__ldg(s)) : 0u, n > 1 ? __float_as_uint(__ldg(s + 1)) : 0u,
                          n > 2 ? __float_as_uint(__ldg(s + 2)) : 0u, 0u);
    } else {
        const uint16_t* s = static_cast<const uint16_t*>(p) + i;
        if (n == 8) return __ldg(reinterpret_cast<const uint4*>(s));
        uint32_t t[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < n) t[e / 2] |= static_cast<uint32_t>(__ldg(s + e)) << (16 * (e & 1));
        return make_uint4(t[0], t[1], t[2], t[3]);
    }
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

template <int XT>
__device__ __forceinline__ void st_vec(void* p, int64_t i, int n, const uint4& q) {
    const uint32_t t[4] = {q.x, q.y, q.z, q.w};
    if constexpr (XT == HQ_F32) {
        float* s = static_cast<float*>(p) + i;
        if (n == 4) {
            *reinterpret_cast<uint4*>(s) = q;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (e < n) s[e] = __uint_as_float(t[e]);
        }
    } else {
        uint16_t* s = static_cast<uint16_t*>(p) + i;
        if (n == 8) {
            *reinterpret_cast<uint4*>(s) = q;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) s[e] = static_cast<uint16_t>(t[e / 2] >> (16 * (e & 1)));
        }
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
            widen<HQ_F32>(ld_vec<HQ_F32>(w, i + h, min(max(n - h, 0), 4)), t);
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
    // (sum of s, max of a) over the CTA
    __device__ __forceinline__ float2 operator()(float s, float a) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            s = __fadd_rn(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
            a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
        }
        const int nw = blockDim.x >> 5;
        if (nw > 1) {
            if ((threadIdx.x & 31) == 0) buf[par][threadIdx.x >> 5] = make_float2(s, a);
            __syncthreads();
            s = 0.f;
            a = 0.f;
            for (int w = 0; w < nw; ++w) {
                const float2 t = buf[par][w];
                s = __fadd_rn(s, t.x);
                a = fmaxf(a, t.y);
            }
            par ^= 1;
        }
        return make_float2(s, a);
    }
};

__device__ __forceinline__ float inv_rms(float sum, int K, float eps) {
    return __frsqrt_rn(__fadd_rn(__fdiv_rn(sum, static_cast<float>(K)), eps));
}

// ---------------------------------------------------------- without a quantiser
// One CTA per row, NV vectors per thread, vector i of thread t at i * threads + t.
// Bound by HBM: everything that a row needs (stream, block, gate, weights) is
// requested before the first reduction, and a row is in registers from then on.
template <int XT, int NV, bool POST, int MAXT>
__global__ void __launch_bounds__(MAXT) k_residual_norm(const NormArgs a) {
    constexpr int V = vec_len<XT>;
    __shared__ float2 red[2][32];
    const int64_t m = blockIdx.x;
    RowReduce reduce{red, 0};
    int col[NV], n[NV];
    uint4 rh[NV], ry[NV], rg[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        col[i] = (i * blockDim.x + threadIdx.x) * V;
        n[i] = min(max(a.K - col[i], 0), V);
        rh[i] = ld_vec<XT>(a.H, m * a.ldh + col[i], n[i]);
    }
    if (a.Y != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i) ry[i] = ld_vec<XT>(a.Y, m * a.ldy + col[i], n[i]);
        if (a.gate != nullptr) {
#pragma unroll
            for (int i = 0; i < NV; ++i) rg[i] = ld_vec<XT>(a.gate, m * a.ldg + col[i], n[i]);
        }
        float rstd = 1.f;
        if constexpr (POST) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float y[V];
                widen<XT>(ry[i], y);
#pragma unroll
                for (int e = 0; e < V; ++e) ss = __fmaf_rn(y[e], y[e], ss);
            }
            rstd = inv_rms(reduce(ss, 0.f).x, a.K, a.eps);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float p[V], h[V];
            widen<XT>(ry[i], p);
            widen<XT>(rh[i], h);
            if constexpr (POST) {
                float w[V];
                ld_weight<V>(a.w_post, a.wt, col[i], n[i], a.off, w);
#pragma unroll
                for (int e = 0; e < V; ++e) p[e] = __fmul_rn(__fmul_rn(p[e], w[e]), rstd);
            }
            if (a.gate != nullptr) {
                float g[V];
                widen<XT>(rg[i], g);
#pragma unroll
                for (int e = 0; e < V; ++e) p[e] = __fmul_rn(g[e], p[e]);
            }
#pragma unroll
            for (int e = 0; e < V; ++e) h[e] = __fadd_rn(h[e], __fmul_rn(a.alpha, p[e]));
            rh[i] = narrow<XT>(h);   // what the norm reads is the stored stream
        }
    }
    if (a.Ho != nullptr) {
#pragma unroll
        for (int i = 0; i < NV; ++i) st_vec<XT>(a.Ho, m * a.ldho + col[i], n[i], rh[i]);
    }
    if (a.w == nullptr) return;   // no norm behind the block
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float h[V];
        widen<XT>(rh[i], h);
#pragma unroll
        for (int e = 0; e < V; ++e) ss = __fmaf_rn(h[e], h[e], ss);
    }
    const float rstd = inv_rms(reduce(ss, 0.f).x, a.K, a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        float h[V], w[V];
        widen<XT>(rh[i], h);
        ld_weight<V>(a.w, a.wt, col[i], n[i], a.off, w);
#pragma unroll
        for (int e = 0; e < V; ++e) h[e] = __fmul_rn(__fmul_rn(h[e], w[e]), rstd);
        st_vec<XT>(a.X, m * a.ldx + col[i], n[i], narrow<XT>(h));
    }
}

// ------------------------------------------------------------- with a quantiser
// One CTA per row; a warp takes 1024 consecutive channels, 32 per thread.  The
// butterfly runs in registers between shared-memory transposes of the warp's
// 1024 fp32 values (a shuffle per element and stage took 4 times the
// shared-memory instructions):
//   layout A: thread l holds channels 256 i + 8 l .. + 7, i = 0..3 (16-byte loads
//             and stores, contiguous over the warp): stages 1, 2, 4
//   layout B: thread l holds channels 256 (l / 8) + l % 8 + 8 k, k = 0..31: stages
//             8 .. 128
//   layout C: thread l holds channels l + 32 q + 256 i, q = 0..7, i = 0..3: stages
//             256, 512 (groups above 256)
//   groups of 2048 and 4096: the 2 or 4 warps of a group exchange the rest in
//             layout C, value by value, through shared memory
// and back to A for the codes.  Channel c of the warp's 1024 is stored at
// c + 8 (c / 256), which makes A's and B's accesses conflict-free (A's 16-byte
// writes two-way).  Only the row's reduction (and the exchange) need the CTA.
constexpr int NQ_SPAN = 1024;
constexpr int NQ_BUF = NQ_SPAN + 32;   // floats per warp

__device__ __forceinline__ float2 f2_add(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 z, x, y;\n\t"
        "mov.b64 {%0, %1}, z;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 f2_sub(float2 a, float2 b) { return f2_add(a, make_float2(-b.x, -b.y)); }

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

template <int XT, int BITS>
__global__ void __launch_bounds__(NM_MAXK / NQ_SPAN * 32) k_norm_quant(const NormArgs a) {
    __shared__ float2 red[2][32];
    extern __shared__ __align__(16) float xch[];   // NQ_BUF per warp
    // the small-M GEMM may be launched early: it waits for this grid's
    // completion before it reads the codes
    asm volatile("griddepcontrol.launch_dependents;");
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.d != nullptr && a.d[0] == -1) record_status(HQ_ERR_ARG);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col0 = warp * NQ_SPAN + lane * 8;
    const int64_t m = blockIdx.x;
    const int G = a.group;
    RowReduce reduce{red, 0};
    float* buf = xch + warp * NQ_BUF;

    // ---- the residual stream after the block, v = h (w + off)
    float v[32];
    float ss = 0.f;
    {
        bool on[4];   // K is a multiple of 32: vectors are whole or absent
        uint4 rh[4], ry[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            on[i] = col0 + 256 * i < a.K;
            rh[i] = on[i] ? ld_vec<XT>(a.H, m * a.ldh + col0 + 256 * i, 8) : make_uint4(0u, 0u, 0u, 0u);
        }
        if (a.Y != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                ry[i] = on[i] ? ld_vec<XT>(a.Y, m * a.ldy + col0 + 256 * i, 8) : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col = col0 + 256 * i;
            float h[8];
            widen<XT>(rh[i], h);
            if (a.Y != nullptr) {
                float p[8];
                widen<XT>(ry[i], p);
                if (a.gate != nullptr && on[i]) {
                    float g[8];
                    widen<XT>(ld_vec<XT>(a.gate, m * a.ldg + col, 8), g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[e] = __fmul_rn(g[e], p[e]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) h[e] = __fadd_rn(h[e], __fmul_rn(a.alpha, p[e]));
                rh[i] = narrow<XT>(h);
                widen<XT>(rh[i], h);   // what the norm reads is the stored stream
            }
            if (a.Ho != nullptr && on[i]) st_vec<XT>(a.Ho, m * a.ldho + col, 8, rh[i]);
            if (on[i]) {
                float w[8];
                ld_weight<8>(a.w, a.wt, col, 8, a.off, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ss = __fmaf_rn(h[e], h[e], ss);
                    v[8 * i + e] = __fmul_rn(h[e], w[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * i + e] = 0.f;
            }
        }
        if (a.X != nullptr) {
            const float rstd = inv_rms(reduce(ss, 0.f).x, a.K, a.eps);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (on[i]) {
                    float x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(v[8 * i + e], rstd);
                    st_vec<XT>(a.X, m * a.ldx + col0 + 256 * i, 8, narrow<XT>(x));
                }
        }
        if (a.d != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int8_t* d = a.d + ((col0 + 256 * i) & (G - 1));
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * i + e] = d[e] == -1 ? -v[8 * i + e] : v[8 * i + e];
            }
        }
    }
    // ---- butterfly, stages in ascending order
    stage<1>(v);
    stage<2>(v);
    stage<4>(v);
    const int ia = 8 * lane, ib = 264 * (lane >> 3) + (lane & 7);   // layouts A (+ 264 i), B (+ 8 k)
    if (G > 8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 8; e += 4)
                *reinterpret_cast<float4*>(buf + ia + 264 * i + e) =
                    make_float4(v[8 * i + e], v[8 * i + e + 1], v[8 * i + e + 2], v[8 * i + e + 3]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = buf[ib + 8 * k];
        stage<1>(v);
        if (G > 16) stage<2>(v);
        if (G > 32) stage<4>(v);
        if (G > 64) stage<8>(v);
        if (G > 128) stage<16>(v);
        if (G > 256) {   // each thread writes where it read
#pragma unroll
            for (int k = 0; k < 32; ++k) buf[ib + 8 * k] = v[k];
            __syncwarp();
            // layout C, element 4 q + i: channel lane + 32 q + 256 i
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = buf[lane + 32 * (k >> 2) + 264 * (k & 3)];
            stage<1>(v);
            if (G > 512) stage<2>(v);
            for (int s = 1; NQ_SPAN * s < G; s <<= 1) {   // partner warp
                const float f = (warp & s) ? -1.f : 1.f;
                const float* other = xch + (warp ^ s) * NQ_BUF;
                if (s > 1) __syncthreads();   // the stage before has been read
#pragma unroll
                for (int k = 0; k < 32; ++k) buf[lane + 32 * (k >> 2) + 264 * (k & 3)] = v[k];
                __syncthreads();
                // the upper warp holds the second term: -own + partner
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = __fmaf_rn(v[k], f, other[lane + 32 * (k >> 2) + 264 * (k & 3)]);
            }
        }
    }
    // ---- row scale; back to layout A
    float amax = 0.f;
#pragma unroll
    for (int k = 0; k < 32; ++k) amax = fmaxf(amax, fabsf(v[k]));
    if (G > NQ_SPAN) __syncthreads();   // the last exchange has been read
    if (G > 256) {
#pragma unroll
        for (int k = 0; k < 32; ++k) buf[lane + 32 * (k >> 2) + 264 * (k & 3)] = v[k];
    } else if (G > 8) {
#pragma unroll
        for (int k = 0; k < 32; ++k) buf[ib + 8 * k] = v[k];
    }
    const float2 t = reduce(ss, amax);
    amax = t.y;
    if (G > 8) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
                const float4 f = *reinterpret_cast<const float4*>(buf + ia + 264 * i + e);
                v[8 * i + e] = f.x; v[8 * i + e + 1] = f.y; v[8 * i + e + 2] = f.z; v[8 * i + e + 3] = f.w;
            }
    }
    constexpr float LEVELS = BITS == 8 ? 127.0f : 7.0f;
    const float inv = amax == 0.f ? 0.f : __fdiv_rn(LEVELS, amax);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (col0 + 256 * i >= a.K) continue;
        const int64_t at = m * a.K + col0 + 256 * i;
        // fl(u * inv) is at most LEVELS (1 + 2^-23): adding 1.5 * 2^23 rounds it
        // to an integer, ties to even, whose two's complement bits end the sum
        uint32_t c[8];
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
            const float2 r = f2_add(make_float2(__fmul_rn(v[8 * i + e], inv), __fmul_rn(v[8 * i + e + 1], inv)),
                                    make_float2(12582912.0f, 12582912.0f));
            c[e] = __float_as_uint(r.x);
            c[e + 1] = __float_as_uint(r.y);
        }
        if constexpr (BITS == 8) {
            const uint32_t lo = __byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410);
            const uint32_t hi = __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410);
            *reinterpret_cast<uint2*>(a.Xq + at) = make_uint2(lo, hi);
        } else {
            uint32_t b = 0u;
#pragma unroll
            for (int e = 0; e < 8; ++e) b |= (c[e] & 0xFu) << (4 * e);
            *reinterpret_cast<uint32_t*>(a.Xq + at / 2) = b;
        }
    }
    // a row with a NaN has a NaN scale, also where nothing else is left of it
    if (threadIdx.x == 0) {
        const float rstd = inv_rms(t.x, a.K, a.eps);
        a.sx[m] = amax == 0.f ? (rstd != rstd ? rstd : 0.f) : __fmul_rn(__fmul_rn(__fdiv_rn(amax, LEVELS), a.cg), rstd);
    }
}

bool nm_al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool nm_type(int t) { return t == HQ_F16 || t == HQ_BF16 || t == HQ_F32; }

template <int XT>
hq_status launch_norm(const NormArgs& a, cudaStream_t st) {
    constexpr int V = vec_len<XT>, NV = XT == HQ_F32 ? 4 : 2;
    const int vecs = (a.K + V - 1) / V;
    const int threads = ((vecs + NV - 1) / NV + 31) / 32 * 32;   // at most 1024
    // up to 512 threads have 128 registers each, which an fp32 row takes
    auto kern = a.w_post != nullptr ? threads <= 512 ? k_residual_norm<XT, NV, true, 512> : k_residual_norm<XT, NV, true, 1024>
                : threads <= 512    ? k_residual_norm<XT, NV, false, 512>
                                    : k_residual_norm<XT, NV, false, 1024>;
    kern<<<static_cast<unsigned>(a.M), threads, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

template <int XT, int BITS>
hq_status launch_norm_quant(const NormArgs& a, cudaStream_t st) {
    const int warps = (a.K + NQ_SPAN - 1) / NQ_SPAN;
    const int smem = warps * NQ_BUF * static_cast<int>(sizeof(float));
    static SmemOptIn opt_in;
    if (!allow_smem(opt_in, k_norm_quant<XT, BITS>, smem)) return HQ_ERR_CUDA;
    k_norm_quant<XT, BITS><<<static_cast<unsigned>(a.M), 32 * warps, smem, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

// Checks shared by the two entry points; the strides are in elements.
hq_status nm_check(const NormArgs& a, int64_t M, int64_t K, int xt) {
    if (M < 0 || K <= 0 || !nm_type(xt) || !nm_type(a.wt) || !(a.eps >= 0.f)) return HQ_ERR_ARG;
    if (M == 0) return HQ_OK;
    if (a.ldh < K || (a.Y && a.ldy < K) || (a.Ho && a.ldho < K) || (a.X && a.ldx < K)) return HQ_ERR_ARG;
    if (a.gate && a.ldg != 0 && a.ldg < K) return HQ_ERR_ARG;
    if (!a.Y && (a.gate || a.w_post)) return HQ_ERR_ARG;
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
    a.cg = static_cast<float>(1.0 / __builtin_sqrt(static_cast<double>(group)));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (xt == HQ_F16) return bits == 8 ? launch_norm_quant<HQ_F16, 8>(a, st) : launch_norm_quant<HQ_F16, 4>(a, st);
    return bits == 8 ? launch_norm_quant<HQ_BF16, 8>(a, st) : launch_norm_quant<HQ_BF16, 4>(a, st);
}
