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
    float* T;          // [M][r_max] in the plan's order
    int64_t ldx;
    int M, K, n, r;
};

constexpr int SH_CL = 8;          // CTAs of a cluster, each a run of K
constexpr int SH_THREADS = 128;
constexpr int SH_STAGES = 5;

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

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
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
    const int q = blockIdx.x;   // rank in the cluster
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
        for (int i = q * SH_THREADS + tid; i < count * RC; i += SH_CL * SH_THREADS)
            if (r0 + i % RC < p.r) p.T[static_cast<int64_t>(start + i / RC) * p.r + r0 + i % RC] = 0.f;
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
    const int lo = static_cast<int>(static_cast<int64_t>(q) * slabs / SH_CL);
    const int hi = static_cast<int>(static_cast<int64_t>(q + 1) * slabs / SH_CL);
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
    for (int i = tid; i < count * RC; i += SH_THREADS) {
        float v = part[i];
#pragma unroll
        for (int w = 1; w < SH_THREADS / 32; ++w) v = __fadd_rn(v, part[w * LR_TILE * RC + i]);
        part[i] = v;
    }
    cluster_sync();
    const float scale = p.scales != nullptr ? p.scales[a] : 1.f;
    for (int i = q * SH_THREADS + tid; i < count * RC; i += SH_CL * SH_THREADS) {
        float v = 0.f;
#pragma unroll
        for (int c = 0; c < SH_CL; ++c) v = __fadd_rn(v, ld_cluster_f32(mapa_shared(smem_u32(part + i), c)));
        const int row = i / RC, col = i % RC;
        if (r0 + col < p.r)
            p.T[static_cast<int64_t>(start + row) * p.r + r0 + col] = col < live ? __fmul_rn(v, scale) : 0.f;
    }
    cluster_sync();   // the partial sums stay until every CTA has read them
}

// ---------------------------------------------------------------------- expand
struct ExpandArgs {
    const float* T;
    const uint16_t* B;
    const int32_t *order, *tiles, *ranks;
    const void* base;
    void* Y;
    int64_t ldb, ldy;
    int M, N, n, r;
};

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t tf32_of(float v) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(v));
    return r;
}

template <int YT>
__device__ __forceinline__ void ex_load8(const void* p, int64_t i, float (&v)[8]) {
    if constexpr (YT == HQ_F32) {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = s[0], b = s[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
        const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        const uint32_t t[4] = {q.x, q.y, q.z, q.w};
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

constexpr int EX_WARPS = 8;
constexpr int EX_COLS = 32 * EX_WARPS;

// A warp takes 32 output columns of a tile.  The product t B^T runs on the tf32
// MMA with t split into two tf32 terms (22 bits) and B, a 16-bit value, exact.
// Both index orders an MMA leaves open are chosen for the loads: within a chunk
// of CH rank positions lane t of a quad holds the CH/4 consecutive ones at
// CH/4 t (one vector load of B and of t), and column c of the i-th n8 tile is
// column 8 (c / 2) + 2 i + c % 2 of the 32, which leaves each lane 8
// consecutive outputs of a row, one 16-byte access of base and of Y.
template <bool BF, int YT, int CH>
__global__ void __launch_bounds__(EX_WARPS * 32) k_lora_expand(const ExpandArgs p) {
    constexpr int PT = CH / 4;   // rank positions per lane and chunk
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    const int n0 = (blockIdx.x * EX_WARPS + warp) * 32;
    const int a = p.tiles[3 * blockIdx.y], start = p.tiles[3 * blockIdx.y + 1], count = p.tiles[3 * blockIdx.y + 2];
    griddep_wait();
    if (count <= 0 || count > LR_TILE || start < 0 || start > p.M - count || a >= p.n || n0 >= p.N) return;
    const int col = n0 + 8 * t4;
    int live = a < 0 ? 0 : p.r;
    if (a >= 0 && p.ranks != nullptr) live = min(max(p.ranks[a], 0), p.r);
    if (live == 0 && p.base == p.Y) return;   // in place: the rows stay as they are
    for (int mt = 0; 16 * mt < count; ++mt) {
        const int i0 = 16 * mt + g;
        int m[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            m[h] = i0 + 8 * h < count ? p.order[start + i0 + 8 * h] : -1;
            if (m[h] >= p.M) m[h] = -1;
        }
        float y[2][8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int e = 0; e < 8; ++e) y[h][e] = 0.f;
            if (p.base != nullptr && m[h] >= 0 && col < p.N) ex_load8<YT>(p.base, m[h] * p.ldb + col, y[h]);
        }
        float acc[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = 0.f;
        for (int c = 0; c * CH < live; ++c) {
            const int j0 = c * CH + PT * t4;   // this lane's first rank position
            float tv[2][PT];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < PT; ++e) tv[h][e] = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (i0 + 8 * h < count) {
                    const float* s = p.T + static_cast<int64_t>(start + i0 + 8 * h) * p.r + j0;
                    if constexpr (PT == 2) {
                        const float2 v = *reinterpret_cast<const float2*>(s);
                        tv[h][0] = v.x; tv[h][1] = v.y;
                    } else {
#pragma unroll
                        for (int e = 0; e < PT; e += 4) {
                            const float4 v = *reinterpret_cast<const float4*>(s + e);
                            tv[h][e] = v.x; tv[h][e + 1] = v.y; tv[h][e + 2] = v.z; tv[h][e + 3] = v.w;
                        }
                    }
                }
            uint32_t bw[4][PT / 2];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int nn = n0 + 8 * (g >> 1) + 2 * i + (g & 1);
#pragma unroll
                for (int e = 0; e < PT / 2; ++e) bw[i][e] = 0u;
                if (nn < p.N) {
                    const uint16_t* s = p.B + (static_cast<int64_t>(a) * p.N + nn) * p.r + j0;
                    if constexpr (PT == 2) {
                        bw[i][0] = __ldg(reinterpret_cast<const uint32_t*>(s));
                    } else if constexpr (PT == 4) {
                        const uint2 v = __ldg(reinterpret_cast<const uint2*>(s));
                        bw[i][0] = v.x; bw[i][1] = v.y;
                    } else {
                        const uint4 v = __ldg(reinterpret_cast<const uint4*>(s));
                        bw[i][0] = v.x; bw[i][1] = v.y; bw[i][2] = v.z; bw[i][3] = v.w;
                    }
                }
            }
#pragma unroll
            for (int s = 0; s < PT / 2; ++s) {   // k = t: position 2 s, k = t + 4: position 2 s + 1
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = tv[e & 1][2 * s + (e >> 1)];
                    hi[e] = tf32_of(v);
                    lo[e] = fabsf(v) < INFINITY ? tf32_of(__fsub_rn(v, __uint_as_float(hi[e]))) : 0u;
                }
                // past the adapter's rank t is zero; B there is not read as a number
                const bool ok0 = j0 + 2 * s < live, ok1 = j0 + 2 * s + 1 < live;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t w = bw[i][s];
                    float b0, b1;
                    if constexpr (BF) {
                        b0 = __uint_as_float(w << 16);
                        b1 = __uint_as_float(w & 0xFFFF0000u);
                    } else {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
                        b0 = f.x;
                        b1 = f.y;
                    }
                    const uint32_t u0 = ok0 ? __float_as_uint(b0) : 0u, u1 = ok1 ? __float_as_uint(b1) : 0u;
                    mma_tf32(acc[i], lo, u0, u1);
                    mma_tf32(acc[i], hi, u0, u1);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (m[h] >= 0 && col < p.N) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (live > 0) {
                        y[h][2 * i] = __fadd_rn(y[h][2 * i], acc[i][2 * h]);
                        y[h][2 * i + 1] = __fadd_rn(y[h][2 * i + 1], acc[i][2 * h + 1]);
                    }
                ex_store8<YT>(p.Y, m[h] * p.ldy + col, y[h]);
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(SH_CL, tiles, (a.r + RC - 1) / RC);
    cfg.blockDim = dim3(SH_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = SH_CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

template <bool BF, int YT>
hq_status launch_expand(const ExpandArgs& a, int tiles, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((a.N + EX_COLS - 1) / EX_COLS, tiles);
    cfg.blockDim = dim3(EX_WARPS * 32);
    cfg.stream = st;
    // may start while k_lora_shrink runs; it waits for that grid's completion
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e;
    if (a.r % 32 == 0)
        e = cudaLaunchKernelEx(&cfg, k_lora_expand<BF, YT, 32>, a);
    else if (a.r % 16 == 0)
        e = cudaLaunchKernelEx(&cfg, k_lora_expand<BF, YT, 16>, a);
    else
        e = cudaLaunchKernelEx(&cfg, k_lora_expand<BF, YT, 8>, a);
    return e == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
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
    s.T = static_cast<float*>(workspace);
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
