// lora.cu -- low-rank adapters of many requests beside a shared projection:
// Y[m] = base[m] + s_a (X[m] A_a^T) B_a^T with a = the adapter of token m, or
// Y[m] = base[m] for a token without one.  `base` is the quantised layer's
// output; X is the layer's 16-bit input, before rotation and quantisation.
//
// The batch's plan (k_lora_plan) sorts the tokens by adapter, stably, and cuts
// the order into tiles of at most 64 tokens of one adapter, so that each
// adapter's matrices are read once per tile and a tile's product is dense.
// k_lora_shrink forms t = s_a X A_a^T (fp32, rank r) per tile, k_lora_expand
// adds t B_a^T to the base rows.  With r <= 64 both are bound by HBM: they do at
// most 2 r flops per element of X and of Y, and X, base and Y are read or
// written once.
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "hq_device.cuh"

namespace hq {
namespace {

constexpr int LR_TILE = 64;         // tokens per tile
constexpr int LR_MAX_ADAPTERS = 1022;   // the plan's CTA has a thread per bucket and one more

__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ------------------------------------------------------------------------ plan
// One CTA: each warp takes a contiguous run of tokens.  Tokens are counted per
// (warp, adapter) in shared memory, the counts scanned in (adapter, warp) order,
// and the tokens placed in their order: the rank of a token among those of the
// same adapter in its group of 32 comes from a warp match.  Bucket 0 holds the
// tokens without an adapter.
constexpr int PL_THREADS = 1024;

__global__ void __launch_bounds__(PL_THREADS) k_lora_plan(const int32_t* __restrict__ ids, int M, int n, int W, int run,
                                                          int32_t* __restrict__ order, int32_t* __restrict__ tiles,
                                                          int max_tiles) {
    extern __shared__ int32_t cnt[];   // [W][n + 1], then begin and first tile per bucket [2][n + 2]
    __shared__ unsigned long long wsum[PL_THREADS / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nb = n + 1;
    int32_t* begin = cnt + W * nb;
    int32_t* first = begin + nb + 1;
    for (int i = tid; i < W * nb; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    auto bucket = [&](int m) {
        const int id = __ldg(ids + m);
        if (id < -1 || id >= n) {
            record_status(HQ_ERR_ARG);
            return 0;
        }
        return id + 1;
    };
    const int lo = warp * run, hi = min(lo + run, M);
    if (warp < W)
        for (int m = lo + lane; m < hi; m += 32) atomicAdd(cnt + warp * nb + bucket(m), 1);
    __syncthreads();
    // thread b: bucket b's total over the warps, then (tokens, tiles) before it
    int total = 0;
    if (tid < nb)
        for (int w = 0; w < W; ++w) {
            const int c = cnt[w * nb + tid];
            cnt[w * nb + tid] = total;
            total += c;
        }
    const unsigned long long mine =
        (static_cast<unsigned long long>(total) << 32) | static_cast<unsigned>((total + LR_TILE - 1) / LR_TILE);
    unsigned long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += t;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    unsigned long long before = inc - mine;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    if (tid <= nb) {   // entry nb: the totals
        begin[tid] = static_cast<int32_t>(before >> 32);
        first[tid] = static_cast<int32_t>(before & 0xFFFFFFFFull);
    }
    if (tid < nb)
        for (int w = 0; w < W; ++w) cnt[w * nb + tid] += static_cast<int32_t>(before >> 32);
    __syncthreads();
    // tiles: the bucket of tile t is the last one whose first tile is <= t
    for (int t = tid; t < max_tiles; t += blockDim.x) {
        int a = -1, s = 0, c = 0;
        if (t < first[nb]) {
            int l = 0, r = nb;
            while (r - l > 1) {
                const int mid = (l + r) >> 1;
                if (first[mid] <= t) l = mid; else r = mid;
            }
            a = l - 1;
            s = begin[l] + (t - first[l]) * LR_TILE;
            c = min(LR_TILE, begin[l + 1] - s);
        }
        tiles[3 * t] = a;
        tiles[3 * t + 1] = s;
        tiles[3 * t + 2] = c;
    }
    if (warp < W)
        for (int m0 = lo; m0 < hi; m0 += 32) {
            const int m = m0 + lane;
            const bool on = m < hi;
            const unsigned act = __ballot_sync(0xFFFFFFFFu, on);
            if (on) {
                const int id = __ldg(ids + m);
                const int b = (id < -1 || id >= n) ? 0 : id + 1;
                const unsigned same = __match_any_sync(act, b);
                const int at = cnt[warp * nb + b];
                order[at + __popc(same & ((1u << lane) - 1u))] = m;
                __syncwarp(act);
                if (lane == __ffs(same) - 1) cnt[warp * nb + b] = at + __popc(same);
            }
            __syncwarp();
        }
}

// ---------------------------------------------------------------------- shrink
struct ShrinkArgs {
    const uint16_t *X, *A;
    const int32_t *order, *tiles, *ranks;
    const float* scales;
    void* T;           // [M][r_max] in the plan's order: fp32, or two bf16 planes
    int64_t ldx;
    int M, K, n, r, planes;
};

constexpr int SH_THREADS = 128;
constexpr int SH_STAGES = 5;
constexpr int SH_MAX_CL = 8;      // CTAs of a cluster, each a run of K

// 8-byte asynchronous global -> shared copy
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}

// 16-byte asynchronous copy; bytes past `bytes` (0 or 16) are written as zero
__device__ __forceinline__ void cp_async16_z(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
                 "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

template <bool BF>
__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
    return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w));
}

__device__ __forceinline__ uint32_t bf16x2_of(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// v as bf16 terms, the first the nearest bf16 and each next one that of the
// rest (zero where the value is not finite: the first term says it all)
__device__ __forceinline__ float bf16_near(float v) { return __bfloat162float(__float2bfloat16_rn(v)); }
__device__ __forceinline__ float rest_of(float v, float near) { return fabsf(near) < INFINITY ? __fsub_rn(v, near) : 0.f; }

// Stores t of four rank positions of one token: fp32, or as two bf16 planes
__device__ __forceinline__ void put_t(const ShrinkArgs& p, int pos, int col, float4 v) {
    const int64_t i = static_cast<int64_t>(pos) * p.r + col;
    if (p.planes == 0) {
        *reinterpret_cast<float4*>(static_cast<float*>(p.T) + i) = v;
    } else {
        uint16_t* t = static_cast<uint16_t*>(p.T);
        const float4 n = make_float4(bf16_near(v.x), bf16_near(v.y), bf16_near(v.z), bf16_near(v.w));
        *reinterpret_cast<uint2*>(t + i) = make_uint2(bf16x2_of(n.x, n.y), bf16x2_of(n.z, n.w));
        *reinterpret_cast<uint2*>(t + i + static_cast<int64_t>(p.M) * p.r) =
            make_uint2(bf16x2_of(rest_of(v.x, n.x), rest_of(v.y, n.y)), bf16x2_of(rest_of(v.z, n.z), rest_of(v.w, n.w)));
    }
}

// One tile and RC columns of the rank per cluster; CTA q of the cluster sums
// its run of K.  Stages of 64 channels stream through a cp.async ring as
// 128-byte rows (16-byte chunk c of row i at chunk c ^ (i & 7)); warp w takes
// channels 16 w .. 16 w + 15 of every stage for all of the tile's tokens, so
// each staged byte is read from shared memory once.  The partial sums meet in
// a fixed order: over the CTA's warps, then over the cluster.
template <bool BF, int RC>
__global__ void __launch_bounds__(SH_THREADS) k_lora_shrink(const ShrinkArgs p) {
    constexpr int STAGE = (LR_TILE + RC) * 128;
    extern __shared__ __align__(128) uint8_t sm[];
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int q = blockIdx.x, cl = gridDim.x;   // rank in the cluster, its CTAs
    const int a = p.tiles[3 * blockIdx.y], start = p.tiles[3 * blockIdx.y + 1], count = p.tiles[3 * blockIdx.y + 2];
    if (a < 0 || count == 0) return;   // no adapter, or an unused tile: the whole cluster leaves
    if (a >= p.n || count < 0 || count > LR_TILE || start < 0 || start > p.M - count) {
        if (tid == 0) record_status(HQ_ERR_ARG);
        return;
    }
    const int r0 = blockIdx.z * RC;
    int live = p.r;
    if (p.ranks != nullptr) {
        live = p.ranks[a];
        if (live < 0 || live > p.r) {
            if (tid == 0) record_status(HQ_ERR_ARG);
            live = live < 0 ? 0 : p.r;
        }
    }
    live = min(max(live - r0, 0), RC);
    if (live == 0) {   // the adapter's rank ends before these columns
        for (int i = q * SH_THREADS + tid; i < count * (RC / 4); i += cl * SH_THREADS) {
            const int row = i / (RC / 4), col = r0 + i % (RC / 4) * 4;
            if (col < p.r) put_t(p, start + row, col, make_float4(0.f, 0.f, 0.f, 0.f));
        }
        return;
    }

    // this thread's rows of a stage: tokens tid/8 + 16 j, adapter rows the same
    const int crow = tid >> 3, chunk = tid & 7;
    const uint16_t* xsrc[LR_TILE / 16];
#pragma unroll
    for (int j = 0; j < LR_TILE / 16; ++j) {
        const int i = crow + 16 * j;
        xsrc[j] = nullptr;
        if (i < count) {
            const int m = p.order[start + i];
            if (m >= 0 && m < p.M)
                xsrc[j] = p.X + m * p.ldx + chunk * 8;
            else
                record_status(HQ_ERR_ARG);
        }
    }
    const uint16_t* asrc = p.A + (static_cast<int64_t>(a) * p.r + r0 + crow) * p.K + chunk * 8;
    const uint32_t ring = smem_u32(sm);
    const uint32_t dst = crow * 128 + ((chunk ^ (crow & 7)) << 4);

    const int slabs = (p.K + 63) / 64;
    const int lo = static_cast<int>(static_cast<int64_t>(q) * slabs / cl);
    const int hi = static_cast<int>(static_cast<int64_t>(q + 1) * slabs / cl);
    auto issue = [&](int s, int slot) {
        if (s < hi) {
            const int k = s * 64;
            const int bytes = k + chunk * 8 < p.K ? 16 : 0;   // K is a multiple of 8
            const uint32_t base = ring + slot * STAGE + dst;
#pragma unroll
            for (int j = 0; j < LR_TILE / 16; ++j)
                if (16 * j < count)   // rows behind the tile are never used
                    cp_async16_z(base + j * 2048, xsrc[j] && bytes ? xsrc[j] + k : p.X, xsrc[j] ? bytes : 0);
#pragma unroll
            for (int j = 0; j < RC / 16; ++j)
                cp_async16_z(base + LR_TILE * 128 + j * 2048,
                             crow + 16 * j < live && bytes ? asrc + static_cast<int64_t>(16 * j) * p.K + k : p.A,
                             crow + 16 * j < live ? bytes : 0);
        }
        cp_async_commit();
    };

    float acc[LR_TILE / 16][RC / 8][4];
#pragma unroll
    for (int mt = 0; mt < LR_TILE / 16; ++mt)
#pragma unroll
        for (int i = 0; i < RC / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][i][e] = 0.f;

    // ldmatrix addresses within a stage: tokens (16 x 16) and adapter rows (two n8 x k16)
    const int am = lane & 15, ac = 2 * warp + (lane >> 4);
    const int bn = (lane & 7) + ((lane >> 4) << 3), bc = 2 * warp + ((lane >> 3) & 1);
    const uint32_t aoff = am * 128 + ((ac ^ (am & 7)) << 4);
    const uint32_t boff = LR_TILE * 128 + bn * 128 + ((bc ^ (bn & 7)) << 4);
    for (int s = 0; s < SH_STAGES - 1; ++s) issue(lo + s, s);
    int slot = 0;
    for (int s = lo; s < hi; ++s) {
        cp_async_wait_group<SH_STAGES - 2>();
        __syncthreads();
        issue(s + SH_STAGES - 1, slot == 0 ? SH_STAGES - 1 : slot - 1);
        const uint32_t st = ring + slot * STAGE;
        uint32_t b[RC / 16][4];
#pragma unroll
        for (int i = 0; i < RC / 16; ++i) ldsm4(b[i], st + boff + i * 2048);
#pragma unroll
        for (int mt = 0; mt < LR_TILE / 16; ++mt)
            if (16 * mt < count) {
                uint32_t x[4];
                ldsm4(x, st + aoff + mt * 2048);
#pragma unroll
                for (int i = 0; i < RC / 16; ++i) {
                    mma_16x8x16<BF>(acc[mt][2 * i], x, b[i][0], b[i][1]);
                    mma_16x8x16<BF>(acc[mt][2 * i + 1], x, b[i][2], b[i][3]);
                }
            }
        slot = slot + 1 == SH_STAGES ? 0 : slot + 1;
    }
    cp_async_wait_all();
    __syncthreads();

    // ---- partial sums: [warp][token][RC], then over the warps into the first
    float* part = reinterpret_cast<float*>(sm);
    const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int mt = 0; mt < LR_TILE / 16; ++mt)
#pragma unroll
        for (int i = 0; i < RC / 8; ++i) {
            float* d = part + (warp * LR_TILE + 16 * mt + g) * RC + 8 * i + 2 * t4;
            *reinterpret_cast<float2*>(d) = make_float2(acc[mt][i][0], acc[mt][i][1]);
            *reinterpret_cast<float2*>(d + 8 * RC) = make_float2(acc[mt][i][2], acc[mt][i][3]);
        }
    __syncthreads();
    float4* part4 = reinterpret_cast<float4*>(sm);
    for (int i = tid; i < count * (RC / 4); i += SH_THREADS) {
        float4 v = part4[i];
#pragma unroll
        for (int w = 1; w < SH_THREADS / 32; ++w) v = add4(v, part4[w * LR_TILE * (RC / 4) + i]);
        part4[i] = v;
    }
    cluster_sync();
    const float scale = p.scales != nullptr ? p.scales[a] : 1.f;
    for (int i = q * SH_THREADS + tid; i < count * (RC / 4); i += cl * SH_THREADS) {
        float4 u[SH_MAX_CL];   // all on their way before the first sum
#pragma unroll
        for (int c = 0; c < SH_MAX_CL; ++c)
            if (c < cl) u[c] = ld_cluster_f32x4(mapa_shared(smem_u32(part4 + i), c));
        float4 v = u[0];
#pragma unroll
        for (int c = 1; c < SH_MAX_CL; ++c)
            if (c < cl) v = add4(v, u[c]);
        const int row = i / (RC / 4), col = i % (RC / 4) * 4;
        v.x = col < live ? __fmul_rn(v.x, scale) : 0.f;
        v.y = col + 1 < live ? __fmul_rn(v.y, scale) : 0.f;
        v.z = col + 2 < live ? __fmul_rn(v.z, scale) : 0.f;
        v.w = col + 3 < live ? __fmul_rn(v.w, scale) : 0.f;
        if (r0 + col < p.r) put_t(p, start + row, r0 + col, v);
    }
    cluster_sync();   // the partial sums stay until every CTA has read them
}

// ---------------------------------------------------------------------- expand
struct ExpandArgs {
    const void* T;
    const uint16_t* B;
    const int32_t *order, *tiles, *ranks;
    const void* base;
    void* Y;
    int64_t ldb, ldy;
    int M, N, n, r;
};

// Eight consecutive outputs as loaded
template <int YT>
struct Out8 {
    uint4 q[YT == HQ_F32 ? 2 : 1];
};

template <int YT>
__device__ __forceinline__ void ex_widen(const Out8<YT>& o, float (&v)[8]) {
    if constexpr (YT == HQ_F32) {
        const uint32_t t[8] = {o.q[0].x, o.q[0].y, o.q[0].z, o.q[0].w, o.q[1].x, o.q[1].y, o.q[1].z, o.q[1].w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(t[e]);
    } else {
        const uint32_t t[4] = {o.q[0].x, o.q[0].y, o.q[0].z, o.q[0].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (YT == HQ_BF16) {
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

template <int YT>
__device__ __forceinline__ void ex_store8(void* p, int64_t i, const float (&v)[8]) {
    if constexpr (YT == HQ_F32) {
        float4* s = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        s[0] = make_float4(v[0], v[1], v[2], v[3]);
        s[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        uint32_t t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (YT == HQ_BF16) {
                const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
                t[e] = *reinterpret_cast<const uint32_t*>(&b);
            } else {
                const __half2 b = __floats2half2_rn(v[2 * e], v[2 * e + 1]);
                t[e] = *reinterpret_cast<const uint32_t*>(&b);
            }
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = make_uint4(t[0], t[1], t[2], t[3]);
    }
}

constexpr int EX_WARPS = 4;
constexpr int EX_COLS = 64 * EX_WARPS;

// A warp takes 64 output columns of a tile.  The product t B^T runs on the
// bf16 MMA with t as two bf16 terms (16-bit Y: 2^-18 of t, far below Y's own
// rounding) or three (fp32 Y), and an fp16 B as its two exact bf16 terms; the
// fp16 MMA would not hold the range of t, and tf32 has a quarter of the rate.
// Both index orders an MMA leaves open are chosen for the loads: within a chunk
// of R rank positions lane t of a quad holds the R/4 consecutive ones from
// R/4 t (vector loads of B and of t), and column c of the i-th of four n8
// tiles is column 8 (c / 2) + 2 i + c % 2 of 32, which leaves each lane 8
// consecutive outputs of a row, one 16-byte access of base and of Y.
template <bool BF, int YT, int R, bool MULTI>
__global__ void __launch_bounds__(EX_WARPS * 32) k_lora_expand(const ExpandArgs p) {
    constexpr int KS = R / 16;               // k16 steps of a chunk
    constexpr int BT = BF ? 1 : 2;           // terms of B
    constexpr int TT = YT == HQ_F32 ? 3 : 2; // terms of t
    extern __shared__ __align__(128) uint8_t sm[];   // t: [term][64][trow], then the base slots
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int n0 = (blockIdx.x * EX_WARPS + warp) * 64;
    const int a = p.tiles[3 * blockIdx.y], start = p.tiles[3 * blockIdx.y + 1], count = p.tiles[3 * blockIdx.y + 2];
    const bool ok = count > 0 && count <= LR_TILE && start >= 0 && start <= p.M - count && a < p.n;
    int live = 0;
    if (ok && a >= 0) live = p.ranks != nullptr ? min(max(p.ranks[a], 0), p.r) : p.r;

    uint32_t b[BT][2][4][KS][2];   // term, 32 columns, n8 tile, k16 step, register
    auto load_b = [&](int c) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int nn = n0 + 32 * w + 8 * (g >> 1) + 2 * i + (g & 1);
                const int j0 = c * R + R / 4 * t4;
                uint32_t v[KS * 2];
#pragma unroll
                for (int e = 0; e < KS * 2; ++e) v[e] = 0u;
                if (nn < p.N) {
                    const uint16_t* s = p.B + (static_cast<int64_t>(a) * p.N + nn) * p.r + j0;
                    if constexpr (R == 16) {
                        if (j0 < live) {
                            const uint2 q = __ldg(reinterpret_cast<const uint2*>(s));
                            v[0] = q.x; v[1] = q.y;
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < KS / 2; ++e)
                            if (j0 + 8 * e < live) {
                                const uint4 q = __ldg(reinterpret_cast<const uint4*>(s) + e);
                                v[4 * e] = q.x; v[4 * e + 1] = q.y; v[4 * e + 2] = q.z; v[4 * e + 3] = q.w;
                            }
                    }
                }
#pragma unroll
                for (int e = 0; e < KS * 2; ++e) {
                    // past the adapter's rank B is not read as a number
                    if (j0 + 2 * e + 1 >= live) v[e] = j0 + 2 * e < live ? v[e] & 0xFFFFu : 0u;
                    if constexpr (BF) {
                        b[0][w][i][e / 2][e & 1] = v[e];
                    } else {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&v[e]));
                        const float h0 = bf16_near(f.x), h1 = bf16_near(f.y);
                        b[0][w][i][e / 2][e & 1] = bf16x2_of(h0, h1);
                        b[BT - 1][w][i][e / 2][e & 1] = bf16x2_of(rest_of(f.x, h0), rest_of(f.y, h1));
                    }
                }
            }
    };
    // this lane's base rows, on their way to slots of its own before t is awaited
    const int rp = (p.r + R - 1) / R * R, trow = 2 * rp + 8;   // bytes of a staged row of t
    uint8_t* slots = sm + TT * LR_TILE * trow + (warp * 32 + lane) * 16;
    constexpr int PIECES = YT == HQ_F32 ? 2 : 1;
    constexpr int SLOT = EX_WARPS * 32 * 16;   // from one piece of a lane to its next
    int m[LR_TILE / 16][2];
#pragma unroll
    for (int mt = 0; mt < LR_TILE / 16; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 16 * mt + 8 * h + g;
            m[mt][h] = ok && i < count ? p.order[start + i] : -1;
            if (m[mt][h] >= p.M) m[mt][h] = -1;
        }
    const bool keep = !ok || (live == 0 && p.base == p.Y);   // nothing to do: in place the rows stay as they are
    if (p.base != nullptr && !keep) {
#pragma unroll
        for (int mt = 0; mt < LR_TILE / 16; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const int col = n0 + 32 * w + 8 * t4;
                    if (m[mt][h] >= 0 && col < p.N) {
                        const uint8_t* src = static_cast<const uint8_t*>(p.base) + (m[mt][h] * p.ldb + col) * (PIECES * 2);
#pragma unroll
                        for (int e = 0; e < PIECES; ++e)
                            cp_async16(smem_u32(slots + (((mt * 2 + h) * 2 + w) * PIECES + e) * SLOT), src + 16 * e);
                    }
                }
    }
    if (!MULTI && live > 0) load_b(0);
    griddep_wait();   // t is complete
    if (live > 0) {   // the same for the whole CTA
        const int64_t plane = static_cast<int64_t>(p.M) * p.r;
        const int per = rp / 4;   // groups of four rank positions
        for (int i = threadIdx.x; i < count * per; i += EX_WARPS * 32) {
            const int row = i / per, j = i % per * 4;
            const int64_t at = static_cast<int64_t>(start + row) * p.r + j;
            uint8_t* dst = sm + row * trow + 2 * j;
            if (j >= p.r) {
#pragma unroll
                for (int e = 0; e < TT; ++e) *reinterpret_cast<uint2*>(dst + e * LR_TILE * trow) = make_uint2(0u, 0u);
            } else if constexpr (YT == HQ_F32) {
                const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(p.T) + at);
                float v[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                for (int e = 0; e < TT; ++e) {
                    const float q[4] = {bf16_near(v[0]), bf16_near(v[1]), bf16_near(v[2]), bf16_near(v[3])};
                    *reinterpret_cast<uint2*>(dst + e * LR_TILE * trow) =
                        make_uint2(bf16x2_of(q[0], q[1]), bf16x2_of(q[2], q[3]));
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[k] = rest_of(v[k], q[k]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < TT; ++e)
                    cp_async8(smem_u32(dst + e * LR_TILE * trow), static_cast<const uint16_t*>(p.T) + e * plane + at);
            }
        }
    }
    cp_async_wait_all();
    __syncthreads();
    if (keep) return;
#pragma unroll
    for (int mt = 0; mt < LR_TILE / 16; ++mt) {
        if (16 * mt >= count) break;
        float acc[2][4][4];
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[w][i][e] = 0.f;
        for (int c = 0; c * R < live; ++c) {
            if (MULTI) load_b(c);
            // small terms first; the product of both last terms is left out
#pragma unroll
            for (int e = TT - 1; e >= 0; --e)
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const uint8_t* src = sm + (e * LR_TILE + 16 * mt + g) * trow + 2 * (c * R + R / 4 * t4 + 4 * s);
                    const uint2 q0 = *reinterpret_cast<const uint2*>(src);
                    const uint2 q1 = *reinterpret_cast<const uint2*>(src + 8 * trow);
                    const uint32_t t[4] = {q0.x, q1.x, q0.y, q1.y};
#pragma unroll
                    for (int f = BT - 1; f >= 0; --f)
                        if (e + f < TT)
#pragma unroll
                            for (int w = 0; w < 2; ++w)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    mma_16x8x16<true>(acc[w][i], t, b[f][w][i][s][0], b[f][w][i][s][1]);
                }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                const int col = n0 + 32 * w + 8 * t4;
                if (m[mt][h] >= 0 && col < p.N) {
                    float v[8] = {};
                    if (p.base != nullptr) {
                        Out8<YT> y;
#pragma unroll
                        for (int e = 0; e < PIECES; ++e)
                            y.q[e] = *reinterpret_cast<const uint4*>(slots + (((mt * 2 + h) * 2 + w) * PIECES + e) * SLOT);
                        ex_widen<YT>(y, v);
                    }
                    if (live > 0) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            v[2 * i] = __fadd_rn(v[2 * i], acc[w][i][2 * h]);
                            v[2 * i + 1] = __fadd_rn(v[2 * i + 1], acc[w][i][2 * h + 1]);
                        }
                    }
                    ex_store8<YT>(p.Y, m[mt][h] * p.ldy + col, v);
                }
            }
    }
}

bool lr_al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <bool BF, int RC>
hq_status launch_shrink(const ShrinkArgs& a, int tiles, cudaStream_t st) {
    constexpr int ring = SH_STAGES * (LR_TILE + RC) * 128, part = SH_THREADS / 32 * LR_TILE * RC * 4;
    constexpr int smem = ring > part ? ring : part;
    auto kern = k_lora_shrink<BF, RC>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return HQ_ERR_CUDA;
    // K is cut as far as one wave of CTAs (two per SM) goes
    const int z = (a.r + RC - 1) / RC;
    const int cl = tiles * z <= 37 ? 8 : tiles * z <= 74 ? 4 : tiles * z <= 148 ? 2 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cl, tiles, z);
    cfg.blockDim = dim3(SH_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cl;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

template <bool BF, int YT, int R, bool MULTI>
hq_status launch_expand_r(const ExpandArgs& a, int tiles, cudaStream_t st) {
    const int rp = (a.r + R - 1) / R * R;
    const int smem = (YT == HQ_F32 ? 3 : 2) * LR_TILE * (2 * rp + 8) + EX_WARPS * 32 * 16 * 16 * (YT == HQ_F32 ? 2 : 1);
    auto kern = k_lora_expand<BF, YT, R, MULTI>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return HQ_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.N + EX_COLS - 1) / EX_COLS, tiles);
    cfg.blockDim = dim3(EX_WARPS * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    // may start while k_lora_shrink runs; it waits for that grid's completion
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

// B's fragments stay in registers for a whole tile where the rank fits: 64
// positions of a 16-bit B used as it is, 32 where B has two terms or t three
template <bool BF, int YT>
hq_status launch_expand(const ExpandArgs& a, int tiles, cudaStream_t st) {
    if (a.r <= 16) return launch_expand_r<BF, YT, 16, false>(a, tiles, st);
    if (a.r <= 32) return launch_expand_r<BF, YT, 32, false>(a, tiles, st);
    if constexpr (BF && YT != HQ_F32) {
        if (a.r <= 64) return launch_expand_r<BF, YT, 64, false>(a, tiles, st);
    }
    return launch_expand_r<BF, YT, 32, true>(a, tiles, st);
}

template <bool BF>
hq_status launch_lora(const ShrinkArgs& s, const ExpandArgs& e, int yt, int tiles, cudaStream_t st) {
    const hq_status r = s.r <= 16 ? launch_shrink<BF, 16>(s, tiles, st)
                        : s.r <= 32 ? launch_shrink<BF, 32>(s, tiles, st)
                                    : launch_shrink<BF, 64>(s, tiles, st);
    if (r != HQ_OK) return r;
    if (yt == HQ_F16) return launch_expand<BF, HQ_F16>(e, tiles, st);
    if (yt == HQ_BF16) return launch_expand<BF, HQ_BF16>(e, tiles, st);
    return launch_expand<BF, HQ_F32>(e, tiles, st);
}

}  // namespace
}  // namespace hq

using namespace hq;

extern "C" int64_t hq_lora_max_tiles(int64_t M, int64_t n) {
    if (M <= 0 || n < 0) return 0;
    return M / LR_TILE + (n + 1 < M ? n + 1 : M);
}

extern "C" hq_status hq_lora_plan(const int32_t* ids, int64_t M, int64_t n, int32_t* order, int32_t* tiles,
                                  void* stream) {
    if (M < 0 || n < 0) return HQ_ERR_ARG;
    if (n > LR_MAX_ADAPTERS || hq_lora_max_tiles(M, n) > 65535) return HQ_ERR_UNSUPPORTED;
    if (M == 0) return HQ_OK;
    if (!ids || !order || !tiles) return HQ_ERR_ARG;
    // a warp per 32 tokens, as far as the counters of its own fit
    const int nb = static_cast<int>(n) + 1;
    int W = static_cast<int>((M + 31) / 32);
    if (W > PL_THREADS / 32) W = PL_THREADS / 32;
    const int run = static_cast<int>(((M + W - 1) / W + 31) / 32 * 32);
    const int smem = (W * nb + 2 * (nb + 1)) * 4;
    // a thread per bucket and one for the totals
    const int threads = 32 * W > nb + 1 ? 32 * W : (nb + 1 + 31) / 32 * 32;
    if (cudaFuncSetAttribute(k_lora_plan, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return HQ_ERR_CUDA;
    k_lora_plan<<<1, threads, smem, static_cast<cudaStream_t>(stream)>>>(
        ids, static_cast<int>(M), static_cast<int>(n), W, run, order, tiles, static_cast<int>(hq_lora_max_tiles(M, n)));
    return cudaGetLastError() == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

extern "C" size_t hq_lora_workspace_size(int64_t M, int32_t r_max) {
    if (M <= 0 || r_max <= 0) return 0;
    return static_cast<size_t>(M) * r_max * sizeof(float);
}

extern "C" hq_status hq_lora_apply(const void* X, hq_dtype xt, int64_t M, int64_t K, int64_t ld_x, const void* A,
                                   const void* B, int64_t N, int64_t n, int32_t r_max, const int32_t* ranks,
                                   const float* scales, const int32_t* order, const int32_t* tiles, const void* base,
                                   int64_t ld_b, void* Y, hq_dtype yt, int64_t ld_y, void* workspace, size_t ws_bytes,
                                   void* stream) {
    if (M < 0 || K <= 0 || N < 0 || n < 0 || r_max <= 0) return HQ_ERR_ARG;
    if (xt != HQ_F16 && xt != HQ_BF16) return xt == HQ_F32 ? HQ_ERR_UNSUPPORTED : HQ_ERR_ARG;
    if (yt != HQ_F16 && yt != HQ_BF16 && yt != HQ_F32) return HQ_ERR_ARG;
    if (ld_x < K || ld_y < N || (base && ld_b < N)) return HQ_ERR_ARG;
    if (base && base == Y && ld_b != ld_y) return HQ_ERR_ARG;
    if (K % 8 != 0 || N % 8 != 0 || r_max % 8 != 0 || r_max > 256) return HQ_ERR_UNSUPPORTED;
    const int64_t n_tiles = hq_lora_max_tiles(M, n);
    if (K > (1 << 24) || N > (1 << 24) || n > LR_MAX_ADAPTERS || n_tiles > 65535) return HQ_ERR_UNSUPPORTED;
    if (M == 0 || N == 0) return HQ_OK;
    if (!X || !Y || !order || !tiles || (n > 0 && (!A || !B))) return HQ_ERR_ARG;
    if (ws_bytes < hq_lora_workspace_size(M, r_max) || !workspace) return HQ_ERR_ARG;
    const int64_t es = yt == HQ_F32 ? 4 : 2;
    if (!lr_al16(X) || !lr_al16(A) || !lr_al16(B) || !lr_al16(Y) || !lr_al16(base) || !lr_al16(workspace) ||
        ld_x * 2 % 16 != 0 || ld_y * es % 16 != 0 || (base && ld_b * es % 16 != 0))
        return HQ_ERR_ALIGN;
    ShrinkArgs s = {};
    s.X = static_cast<const uint16_t*>(X);
    s.A = static_cast<const uint16_t*>(A);
    s.order = order; s.tiles = tiles; s.ranks = ranks; s.scales = scales;
    s.T = workspace;
    s.planes = yt == HQ_F32 ? 0 : 2;
    s.ldx = ld_x;
    s.M = static_cast<int>(M); s.K = static_cast<int>(K); s.n = static_cast<int>(n); s.r = r_max;
    ExpandArgs e = {};
    e.T = s.T;
    e.B = static_cast<const uint16_t*>(B);
    e.order = order; e.tiles = tiles; e.ranks = ranks;
    e.base = base; e.Y = Y; e.ldb = ld_b; e.ldy = ld_y;
    e.M = s.M; e.N = static_cast<int>(N); e.n = s.n; e.r = r_max;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return xt == HQ_BF16 ? launch_lora<true>(s, e, yt, static_cast<int>(n_tiles), st)
                         : launch_lora<false>(s, e, yt, static_cast<int>(n_tiles), st);
}
