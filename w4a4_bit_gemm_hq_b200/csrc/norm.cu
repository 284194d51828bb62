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

constexpr int NM_NV = 4;              // 8-channel vectors per thread
constexpr int NM_SPAN = 256 * NM_NV;  // channels per warp
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

template <int XT>
struct Raw {   // eight stream values as loaded
    uint4 q[XT == HQ_F32 ? 2 : 1];
};

template <int XT>
__device__ __forceinline__ Raw<XT> ld_raw(const void* p, int64_t i, int n) {
    Raw<XT> r;
    if constexpr (XT == HQ_F32) {
        const float* s = static_cast<const float*>(p) + i;
        if (n == 8) {
            r.q[0] = __ldg(reinterpret_cast<const uint4*>(s));
            r.q[1] = __ldg(reinterpret_cast<const uint4*>(s) + 1);
        } else {
            uint32_t t[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) t[e] = e < n ? __float_as_uint(__ldg(s + e)) : 0u;
            r.q[0] = make_uint4(t[0], t[1], t[2], t[3]);
            r.q[1] = make_uint4(t[4], t[5], t[6], t[7]);
        }
    } else {
        const uint16_t* s = static_cast<const uint16_t*>(p) + i;
        if (n == 8) {
            r.q[0] = __ldg(reinterpret_cast<const uint4*>(s));
        } else {
            uint32_t t[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) t[e / 2] |= static_cast<uint32_t>(__ldg(s + e)) << (16 * (e & 1));
            r.q[0] = make_uint4(t[0], t[1], t[2], t[3]);
        }
    }
    return r;
}

template <int XT>
__device__ __forceinline__ void widen(const Raw<XT>& r, float (&v)[8]) {
    if constexpr (XT == HQ_F32) {
        const uint32_t t[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w, r.q[1].x, r.q[1].y, r.q[1].z, r.q[1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(t[e]);
    } else {
        const uint32_t t[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (XT == HQ_BF16) {
                v[2 * e] = __uint_as_float(t[e] << 16);
                v[2 * e + 1] = __uint_as_float(t[e] & 0xFFFF0000u);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&t[e]));
                v[2 * e] = f.x;
                v[2 * e + 1] = f.y;
            }
        }
    }
}

template <int XT>
__device__ __forceinline__ Raw<XT> narrow(const float (&v)[8]) {
    Raw<XT> r;
    uint32_t t[8];
    if constexpr (XT == HQ_F32) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = __float_as_uint(v[e]);
        r.q[0] = make_uint4(t[0], t[1], t[2], t[3]);
        r.q[1] = make_uint4(t[4], t[5], t[6], t[7]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (XT == HQ_BF16) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                t[e] = *reinterpret_cast<const uint32_t*>(&b);
            } else {
                const __half2 b = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
                t[e] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
        r.q[0] = make_uint4(t[0], t[1], t[2], t[3]);
    }
    return r;
}

template <int XT>
__device__ __forceinline__ void st_raw(void* p, int64_t i, int n, const Raw<XT>& r) {
    if constexpr (XT == HQ_F32) {
        float* s = static_cast<float*>(p) + i;
        if (n == 8) {
            reinterpret_cast<uint4*>(s)[0] = r.q[0];
            reinterpret_cast<uint4*>(s)[1] = r.q[1];
        } else {
            const uint32_t t[8] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w, r.q[1].x, r.q[1].y, r.q[1].z, r.q[1].w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) s[e] = __uint_as_float(t[e]);
        }
    } else {
        uint16_t* s = static_cast<uint16_t*>(p) + i;
        if (n == 8) {
            *reinterpret_cast<uint4*>(s) = r.q[0];
        } else {
            const uint32_t t[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (e < n) s[e] = static_cast<uint16_t>(t[e / 2] >> (16 * (e & 1)));
        }
    }
}

// eight norm weights plus the offset; their type is a run-time choice (the
// branch is the same for the whole grid)
__device__ __forceinline__ void ld_weight(const void* w, int wt, int i, int n, float off, float (&v)[8]) {
    if (wt == HQ_F32)
        widen<HQ_F32>(ld_raw<HQ_F32>(w, i, n), v);
    else if (wt == HQ_BF16)
        widen<HQ_BF16>(ld_raw<HQ_BF16>(w, i, n), v);
    else
        widen<HQ_F16>(ld_raw<HQ_F16>(w, i, n), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __fadd_rn(v[e], off);
}

// Row-wide reductions: sums and maxima over the CTA in a fixed order, one
// barrier each.  Two buffers used in turn: a buffer is written again only after
// the next reduction's barrier, which every thread reaches after reading it.
struct RowReduce {
    float2 (*buf)[NM_MAXK / NM_SPAN];
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

// Thread (warp w, lane l) holds the vectors of channels w * 1024 + i * 256 +
// 8 l .. + 7, i = 0..3: loads and stores are contiguous over a warp, butterfly
// stages 1..4 run inside a vector, 8..128 across lanes, 256 and 512 across the
// thread's vectors, 1024 and 2048 across warps through shared memory.
template <int XT, int BITS, bool POST>
__global__ void __launch_bounds__(NM_MAXK / NM_SPAN * 32) k_norm(const NormArgs a) {
    __shared__ float2 red[2][NM_MAXK / NM_SPAN];
    extern __shared__ float xch[];   // 32 floats per thread, groups of 2048 and more
    if constexpr (BITS != 0) {
        // the small-M GEMM may be launched early: it waits for this grid's
        // completion before it reads the codes
        asm volatile("griddepcontrol.launch_dependents;");
        if (blockIdx.x == 0 && threadIdx.x == 0 && a.d != nullptr && a.d[0] == -1) record_status(HQ_ERR_ARG);
    }
    const int lane = threadIdx.x & 31;
    const int col0 = (threadIdx.x >> 5) * NM_SPAN + lane * 8;
    const int64_t m = blockIdx.x;
    RowReduce reduce{red, 0};

    int n[NM_NV];
    float h[NM_NV][8];
#pragma unroll
    for (int i = 0; i < NM_NV; ++i) {
        const int left = a.K - (col0 + 256 * i);
        n[i] = left < 0 ? 0 : left < 8 ? left : 8;
    }
    // ---- the residual stream after the block
    {
        Raw<XT> rh[NM_NV], ry[NM_NV];
#pragma unroll
        for (int i = 0; i < NM_NV; ++i) rh[i] = ld_raw<XT>(a.H, m * a.ldh + col0 + 256 * i, n[i]);
        if (a.Y != nullptr) {
#pragma unroll
            for (int i = 0; i < NM_NV; ++i) ry[i] = ld_raw<XT>(a.Y, m * a.ldy + col0 + 256 * i, n[i]);
        }
        float rstd = 1.f;
        if constexpr (POST) {
            float ss = 0.f;
#pragma unroll
            for (int i = 0; i < NM_NV; ++i) {
                float y[8];
                widen<XT>(ry[i], y);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = __fmaf_rn(y[e], y[e], ss);
            }
            rstd = inv_rms(reduce(ss, 0.f).x, a.K, a.eps);
        }
#pragma unroll
        for (int i = 0; i < NM_NV; ++i) {
            widen<XT>(rh[i], h[i]);
            if (a.Y != nullptr) {
                float p[8];
                widen<XT>(ry[i], p);
                if constexpr (POST) {
                    float w[8];
                    ld_weight(a.w_post, a.wt, col0 + 256 * i, n[i], a.off, w);
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[e] = __fmul_rn(__fmul_rn(p[e], w[e]), rstd);
                }
                if (a.gate != nullptr) {
                    float g[8];
                    widen<XT>(ld_raw<XT>(a.gate, m * a.ldg + col0 + 256 * i, n[i]), g);
#pragma unroll
                    for (int e = 0; e < 8; ++e) p[e] = __fmul_rn(g[e], p[e]);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] = __fadd_rn(h[i][e], __fmul_rn(a.alpha, p[e]));
                const Raw<XT> r = narrow<XT>(h[i]);
                widen<XT>(r, h[i]);   // what the norm reads is the stored stream
                if (a.Ho != nullptr) st_raw<XT>(a.Ho, m * a.ldho + col0 + 256 * i, n[i], r);
            } else if (a.Ho != nullptr) {
                st_raw<XT>(a.Ho, m * a.ldho + col0 + 256 * i, n[i], rh[i]);
            }
        }
    }
    if (a.w == nullptr) return;   // no norm behind the block

    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NM_NV; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = __fmaf_rn(h[i][e], h[i][e], ss);
        float w[8];
        ld_weight(a.w, a.wt, col0 + 256 * i, n[i], a.off, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = n[i] > 0 ? __fmul_rn(h[i][e], w[e]) : 0.f;   // v from here on
    }
    float rstd = 0.f;
    if (BITS == 0 || a.X != nullptr) {
        rstd = inv_rms(reduce(ss, 0.f).x, a.K, a.eps);
#pragma unroll
        for (int i = 0; i < NM_NV; ++i) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(h[i][e], rstd);
            st_raw<XT>(a.X, m * a.ldx + col0 + 256 * i, n[i], narrow<XT>(x));
        }
    }
    if constexpr (BITS != 0) {
        const int G = a.group;
        if (a.d != nullptr) {
#pragma unroll
            for (int i = 0; i < NM_NV; ++i)
                if (n[i] > 0) {
                    const int8_t* d = a.d + ((col0 + 256 * i) & (G - 1));
#pragma unroll
                    for (int e = 0; e < 8; ++e) h[i][e] = d[e] == -1 ? -h[i][e] : h[i][e];
                }
        }
        // ---- butterfly, stages in ascending order
#pragma unroll
        for (int s = 1; s < 8; s <<= 1)
#pragma unroll
            for (int i = 0; i < NM_NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if ((e & s) == 0) {
                        const float p = h[i][e], q = h[i][e + s];
                        h[i][e] = __fadd_rn(p, q);
                        h[i][e + s] = __fsub_rn(p, q);
                    }
#pragma unroll
        for (int s = 1; s < 32; s <<= 1)
            if (8 * s < G) {
                // the upper lane holds the second term: -own + partner
                const float f = (lane & s) ? -1.f : 1.f;
#pragma unroll
                for (int i = 0; i < NM_NV; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        h[i][e] = __fmaf_rn(h[i][e], f, __shfl_xor_sync(0xFFFFFFFFu, h[i][e], s));
            }
#pragma unroll
        for (int s = 1; s < NM_NV; s <<= 1)
            if (256 * s < G) {
#pragma unroll
                for (int i = 0; i < NM_NV; ++i)
                    if ((i & s) == 0) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float p = h[i][e], q = h[i + s][e];
                            h[i][e] = __fadd_rn(p, q);
                            h[i + s][e] = __fsub_rn(p, q);
                        }
                    }
            }
        for (int s = 1; NM_SPAN * s < G; s <<= 1) {   // partner warp
            const int t = threadIdx.x, nt = blockDim.x;
            const float f = ((t >> 5) & s) ? -1.f : 1.f;
            if (s > 1) __syncthreads();   // the stage before has been read
#pragma unroll
            for (int i = 0; i < NM_NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) xch[(8 * i + e) * nt + t] = h[i][e];
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NM_NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    h[i][e] = __fmaf_rn(h[i][e], f, xch[(8 * i + e) * nt + (t ^ (32 * s))]);
        }
        // ---- row scale, codes
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < NM_NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(h[i][e]));
        const float2 t = reduce(ss, amax);
        if (a.X == nullptr) rstd = inv_rms(t.x, a.K, a.eps);
        amax = t.y;
        constexpr float LEVELS = BITS == 8 ? 127.0f : 7.0f;
        const float inv = amax == 0.f ? 0.f : __fdiv_rn(LEVELS, amax);
#pragma unroll
        for (int i = 0; i < NM_NV; ++i) {
            if (n[i] <= 0) continue;
            const int64_t at = m * a.K + col0 + 256 * i;
            // fl(u * inv) is at most LEVELS (1 + 2^-23): adding 1.5 * 2^23 rounds it
            // to an integer, ties to even, whose two's complement bits end the sum
            if constexpr (BITS == 8) {
                uint32_t b[2] = {0u, 0u};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    b[e / 4] |= (__float_as_uint(__fadd_rn(__fmul_rn(h[i][e], inv), 12582912.0f)) & 0xFFu) << (8 * (e & 3));
                *reinterpret_cast<uint2*>(a.Xq + at) = make_uint2(b[0], b[1]);
            } else {
                uint32_t b = 0u;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    b |= (__float_as_uint(__fadd_rn(__fmul_rn(h[i][e], inv), 12582912.0f)) & 0xFu) << (4 * e);
                *reinterpret_cast<uint32_t*>(a.Xq + at / 2) = b;
            }
        }
        // a row with a NaN has a NaN scale, also where nothing else is left of it
        if (threadIdx.x == 0)
            a.sx[m] = amax == 0.f ? (rstd != rstd ? rstd : 0.f)
                                  : __fmul_rn(__fmul_rn(__fdiv_rn(amax, LEVELS), a.cg), rstd);
    }
}

bool nm_al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool nm_type(int t) { return t == HQ_F16 || t == HQ_BF16 || t == HQ_F32; }

template <int XT, int BITS>
hq_status nm_launch(const NormArgs& a, cudaStream_t st) {
    const int threads = (a.K + NM_SPAN - 1) / NM_SPAN * 32;
    const size_t shm = a.group > NM_SPAN ? static_cast<size_t>(threads) * 32 * sizeof(float) : 0;
    auto run = [&](auto kern) -> hq_status {
        static SmemOptIn opt_in;   // of the one kernel of this instance that takes any (BITS != 0)
        if (!allow_smem(opt_in, kern, static_cast<int>(shm))) return HQ_ERR_CUDA;
        kern<<<static_cast<unsigned>(a.M), threads, shm, st>>>(a);
        return cudaGetLastError() == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
    };
    if constexpr (BITS == 0) {
        if (a.w_post != nullptr) return run(k_norm<XT, 0, true>);
    }
    return run(k_norm<XT, BITS, false>);
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
    if (xt == HQ_F16) return nm_launch<HQ_F16, 0>(a, st);
    if (xt == HQ_BF16) return nm_launch<HQ_BF16, 0>(a, st);
    return nm_launch<HQ_F32, 0>(a, st);
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
    if (xt == HQ_F16) return bits == 8 ? nm_launch<HQ_F16, 8>(a, st) : nm_launch<HQ_F16, 4>(a, st);
    return bits == 8 ? nm_launch<HQ_BF16, 8>(a, st) : nm_launch<HQ_BF16, 4>(a, st);
}
