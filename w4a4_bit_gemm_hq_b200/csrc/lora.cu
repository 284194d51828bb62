// lora.cu -- low-rank adapters of many requests beside a shared projection:
// Y[m] = base[m] + s_a (X[m] A_a^T) B_a^T with a = the adapter of token m, or
// Y[m] = base[m] for a token without one.  `base` is the quantised layer's
// output; X is the layer's 16-bit input, before rotation and quantisation.
//
// The batch's plan (k_lora_plan) sorts the tokens by adapter, stably, and cuts
// the order into tiles of at most 64 tokens of one adapter, so that each
// adapter's matrices are read once per tile and a tile's product is dense.
// k_lora_shrink forms t = s_a X A_a^T (fp32, rank r) per tile, k_lora_expand
// adds t B_a^T to the base rows; where the batch has fewer than 16 tokens for each
// tile that its plan may hold (decode; also prompts beside many resident adapters,
// see launch_lora_y) k_lora_few does both in one launch.  They do at most 2 r flops
// per element of X and of Y, so for r <= 64 the floor is HBM's: X, base and Y once,
// and the matrices of the adapters in use.  Measured, GPU time: 1 token 4096 ->
// 11008, rank 16: 5.9 us; 16 tokens of 16 adapters, rank 32: 9.4 us (1.4 at HBM's
// rate); 2048 x 4096 -> 4096, rank 32: 24.8 us (7.8); 8192 x 8192 -> 28672, rank 64:
// 242 us (170).  Above rank 64 the shrink reads X once for every 64 rank positions:
// 2048 x 4096 -> 4096, rank 128 45 us (10); 8192 x 4096 -> 11008, rank 256 208 us (70).
// Accumulators are the tensor cores' fp32, which truncates, but plain fp32 in the
// second product of the few-token forms: the last bits of a token may differ with the
// batch it comes in.
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "hq_device.cuh"

namespace hq {
namespace {

constexpr int LR_TILE = 64;         // tokens per tile
constexpr int LR_MAX_ADAPTERS = 1022;   // the plan's CTA has a thread per bucket and one more

// Where part q of cl (a power of two) of `n` (below 2^24) begins
__device__ __forceinline__ int part_of(int n, int q, int cl) { return (q * n) >> (__ffs(cl) - 1); }

__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ------------------------------------------------------------------------ plan
// A cluster of CTAs (one for short batches), each a contiguous run of tokens, and
// each warp of a CTA a run of that.  Tokens are counted per (warp, adapter) in
// shared memory, the counts scanned in (adapter, CTA, warp) order, and the tokens
// placed in their order: the rank of a token among those of the same adapter in
// its group of 32 comes from a warp match.  Bucket 0 holds the tokens without an
// adapter.  Bound by the latency of these steps, not by its few bytes (16 tokens 2.7
// us, 32768 tokens 7.3 us; one CTA for all of those took 21).
constexpr int PL_THREADS = 1024;
constexpr int PL_RUN = 4096;        // tokens of a CTA before another one is added
constexpr int PL_MAX_CL = 8;

__global__ void __launch_bounds__(PL_THREADS) k_lora_plan(const int32_t* __restrict__ ids, int M, int n, int W, int run,
                                                          int32_t* __restrict__ order, int32_t* __restrict__ tiles,
                                                          int max_tiles) {
    extern __shared__ int32_t cnt[];   // [W][nb]; begin and first tile per bucket [2][nb + 1]; tokens per bucket [nb]
    __shared__ unsigned long long wsum[PL_THREADS / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = blockIdx.x, cl = gridDim.x;
    const int nb = n + 1;
    int32_t* begin = cnt + W * nb;
    int32_t* first = begin + nb + 1;
    int32_t* mine = first + nb + 1;
    for (int i = tid; i < W * nb; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    auto bucket = [&](int id) { return id < -1 || id >= n ? 0 : id + 1; };
    const int lo = (rank * W + warp) * run, hi = min(lo + run, M);
    bool bad = false;
    if (warp < W)
        for (int m0 = lo; m0 < hi; m0 += 128) {   // four loads on their way at a time
            int id[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) id[k] = m0 + 32 * k + lane < hi ? __ldg(ids + m0 + 32 * k + lane) : -1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                bad |= id[k] < -1 || id[k] >= n;
                if (m0 + 32 * k + lane < hi) atomicAdd(cnt + warp * nb + bucket(id[k]), 1);
            }
        }
    if (bad) record_status(HQ_ERR_ARG);
    __syncthreads();
    // thread b: bucket b's tokens in this CTA, over its warps
    int total = 0;
    if (tid < nb) {
        for (int w = 0; w < W; ++w) {
            const int c = cnt[w * nb + tid];
            cnt[w * nb + tid] = total;
            total += c;
        }
        mine[tid] = total;
    }
    int ahead = 0;   // bucket b's tokens in the CTAs before this one
    if (cl > 1) {
        cluster_sync();
        total = 0;
        if (tid < nb)
            for (int c = 0; c < cl; ++c) {
                int32_t v;
                asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(mine + tid), c)) : "memory");
                if (c < rank) ahead += v;
                total += v;
            }
    }
    // (tokens, tiles) before bucket b
    const unsigned long long own =
        (static_cast<unsigned long long>(total) << 32) | static_cast<unsigned>((total + LR_TILE - 1) / LR_TILE);
    unsigned long long inc = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long t = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += t;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    unsigned long long before = inc - own;
    for (int w = 0; w < warp; ++w) before += wsum[w];
    if (tid <= nb) {   // entry nb: the totals
        begin[tid] = static_cast<int32_t>(before >> 32);
        first[tid] = static_cast<int32_t>(before & 0xFFFFFFFFull);
    }
    if (tid < nb)
        for (int w = 0; w < W; ++w) cnt[w * nb + tid] += static_cast<int32_t>(before >> 32) + ahead;
    __syncthreads();
    if (warp < W)
        for (int m0 = lo; m0 < hi; m0 += 128) {
            int b[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)   // lanes behind the end form a bucket of their own
                b[k] = m0 + 32 * k + lane < hi ? bucket(__ldg(ids + m0 + 32 * k + lane)) : -1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const unsigned same = __match_any_sync(0xFFFFFFFFu, b[k]);
                const int at = b[k] >= 0 ? cnt[warp * nb + b[k]] : 0;
                __syncwarp();
                if (b[k] >= 0) {
                    order[at + __popc(same & ((1u << lane) - 1u))] = m0 + 32 * k + lane;
                    if (lane == __ffs(same) - 1) cnt[warp * nb + b[k]] = at + __popc(same);
                }
                __syncwarp();
            }
        }
    // tiles: the bucket of tile t is the last one whose first tile is <= t
    for (int t = rank * blockDim.x + tid; t < max_tiles; t += cl * blockDim.x) {
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
    if (cl > 1) cluster_sync();   // the counts stay until every CTA has read them
}

// ---------------------------------------------------------------------- shrink
__device__ __forceinline__ void prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<uint64_t>(p)));
}

struct ShrinkArgs {
    const uint16_t *X, *A;
    const int32_t *order, *tiles, *ranks;
    const float* scales;
    float* T;          // [M][r_max] in the plan's order
    int64_t ldx;
    int M, K, n, r;
};

constexpr int SH_THREADS = 256;
constexpr int SH_STAGES = 3;
constexpr int SH_MAX_CL = 8;      // CTAs of a cluster, each a run of K
// CTAs per SM that registers and shared memory are sized for
template <int RC>
constexpr int sh_ctas = RC == 64 ? 2 : 3;

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

// What a thread needs of tile i: the tile, its adapter's rank, and the tokens
// whose rows the thread copies (tid / 16 + 16 j of the tile, -1 for none).  Two
// dependent loads in all: the rank and the tokens are asked for together.  False
// where there is nothing to do (no adapter, an unused or a bad entry).
struct ShrinkTile {
    int a, start, count, live;
    int m[LR_TILE / 16];
};

__device__ __forceinline__ bool shrink_tile(const ShrinkArgs& p, int i, ShrinkTile& t) {
    t.a = p.tiles[3 * i];
    t.start = p.tiles[3 * i + 1];
    t.count = p.tiles[3 * i + 2];
    if (t.a < 0 || t.count == 0) return false;
    if (t.a >= p.n || t.count < 0 || t.count > LR_TILE || t.start < 0 || t.start > p.M - t.count) {
        if (threadIdx.x == 0) record_status(HQ_ERR_ARG);
        return false;
    }
    const int row = threadIdx.x < SH_THREADS ? threadIdx.x >> 4 : LR_TILE;   // the others have none
#pragma unroll
    for (int j = 0; j < LR_TILE / 16; ++j) t.m[j] = row + 16 * j < t.count ? p.order[t.start + row + 16 * j] : 0;
    t.live = p.ranks != nullptr ? p.ranks[t.a] : p.r;
    bool bad = t.live < 0 || t.live > p.r;
    t.live = min(max(t.live, 0), p.r);
#pragma unroll
    for (int j = 0; j < LR_TILE / 16; ++j)
        if (t.m[j] < 0 || t.m[j] >= p.M) {
            bad = true;
            t.m[j] = -1;
        }
    if (bad) record_status(HQ_ERR_ARG);
#pragma unroll
    for (int j = 0; j < LR_TILE / 16; ++j)
        if (row + 16 * j >= t.count) t.m[j] = -1;
    return true;
}

// The sums of one tile and RC columns of the rank over CTA q's part of K (of cl
// parts), left in `sm` as [token][RC].  Stages of 128 channels stream through a
// cp.async ring as two halves of 128-byte rows (16-byte chunk c of row i at
// chunk c ^ (i & 7)).  Warp (h, w) takes 32 of the tile's tokens and channels
// 16 w .. 16 w + 15 of each half; the warps' sums meet in a fixed order.
// For the first SH_THREADS threads of a CTA; the others of `ALL` wait on barrier 2
// until the first stages have been asked for.
template <bool BF, int RC, int ALL>
__device__ __forceinline__ void shrink_part(const ShrinkArgs& p, const ShrinkTile& t, int r0, int live, int q, int cl,
                                            uint8_t* sm) {
    constexpr int HALF = (LR_TILE + RC) * 128, STAGE = 2 * HALF;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // this thread's rows of a stage: tokens tid/16 + 16 j, adapter rows the same
    const int count = t.count, crow = tid >> 4, chunk = tid & 15;
    const uint16_t* xsrc[LR_TILE / 16];
#pragma unroll
    for (int j = 0; j < LR_TILE / 16; ++j) xsrc[j] = t.m[j] >= 0 ? p.X + t.m[j] * p.ldx + chunk * 8 : nullptr;
    const uint16_t* asrc = p.A + (static_cast<int64_t>(t.a) * p.r + r0 + crow) * p.K + chunk * 8;
    const uint32_t ring = smem_u32(sm);
    const uint32_t dst = (chunk >> 3) * HALF + crow * 128 + (((chunk & 7) ^ (crow & 7)) << 4);

    const int slabs = (p.K + 127) / 128;
    const int lo = part_of(slabs, q, cl), hi = part_of(slabs, q + 1, cl);
    auto issue = [&](int s, int slot) {
        if (s < hi) {
            const int k = s * 128;
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

    float acc[2][RC / 8][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < RC / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][i][e] = 0.f;

    // ldmatrix addresses within half a stage: tokens (16 x 16) and adapter rows (two n8 x k16)
    const int wk = warp & 3, m0 = (warp >> 2) * 32;
    const int am = lane & 15, ac = 2 * wk + (lane >> 4);
    const int bn = (lane & 7) + ((lane >> 4) << 3), bc = 2 * wk + ((lane >> 3) & 1);
    const uint32_t aoff = (m0 + am) * 128 + ((ac ^ (am & 7)) << 4);
    const uint32_t boff = LR_TILE * 128 + bn * 128 + ((bc ^ (bn & 7)) << 4);
    for (int s = 0; s < SH_STAGES - 1; ++s) issue(lo + s, s);
    if constexpr (ALL > SH_THREADS) asm volatile("bar.arrive 2, %0;" ::"n"(ALL) : "memory");
    int slot = 0;
    for (int s = lo; s < hi; ++s) {
        cp_async_wait_group<SH_STAGES - 2>();
        named_bar_sync(1, SH_THREADS);
        issue(s + SH_STAGES - 1, slot == 0 ? SH_STAGES - 1 : slot - 1);
        if (m0 < count) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t st = ring + slot * STAGE + h * HALF;
                uint32_t x[2][4];
                ldsm4(x[0], st + aoff);
                if (m0 + 16 < count) ldsm4(x[1], st + aoff + 2048);
#pragma unroll
                for (int i = 0; i < RC / 16; ++i) {
                    uint32_t b[4];
                    ldsm4(b, st + boff + i * 2048);
#pragma unroll
                    for (int mt = 0; mt < 2; ++mt)
                        if (mt == 0 || m0 + 16 < count) {
                            mma_16x8x16<BF>(acc[mt][2 * i], x[mt], b[0], b[1]);
                            mma_16x8x16<BF>(acc[mt][2 * i + 1], x[mt], b[2], b[3]);
                        }
                }
            }
        }
        slot = slot + 1 == SH_STAGES ? 0 : slot + 1;
    }
    cp_async_wait_all();
    named_bar_sync(1, SH_THREADS);

    // ---- partial sums: [k16 warp][token][RC], then over those warps into the first
    float* part = reinterpret_cast<float*>(sm);
    const int g = lane >> 2, t4 = lane & 3;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int i = 0; i < RC / 8; ++i) {
            float* d = part + (wk * LR_TILE + m0 + 16 * mt + g) * RC + 8 * i + 2 * t4;
            *reinterpret_cast<float2*>(d) = make_float2(acc[mt][i][0], acc[mt][i][1]);
            *reinterpret_cast<float2*>(d + 8 * RC) = make_float2(acc[mt][i][2], acc[mt][i][3]);
        }
    named_bar_sync(1, SH_THREADS);
    float4* part4 = reinterpret_cast<float4*>(sm);
    for (int i = tid; i < count * (RC / 4); i += SH_THREADS) {
        float4 v = part4[i];
#pragma unroll
        for (int w = 1; w < 4; ++w) v = add4(v, part4[w * LR_TILE * (RC / 4) + i]);
        part4[i] = v;
    }
}

// One tile and RC columns of the rank per cluster, CTA q a part of K; the partial
// sums meet in a fixed order over the cluster.
template <bool BF, int RC>
__global__ void __launch_bounds__(SH_THREADS, sh_ctas<RC>) k_lora_shrink(const ShrinkArgs p) {
    extern __shared__ __align__(128) uint8_t sm[];
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x;
    const int q = blockIdx.x, cl = gridDim.x;   // rank in the cluster, its CTAs
    ShrinkTile t;
    if (!shrink_tile(p, blockIdx.y, t)) return;   // the whole cluster leaves
    const int start = t.start, count = t.count;
    const int r0 = blockIdx.z * RC, live = min(max(t.live - r0, 0), RC);
    if (live == 0) {   // the adapter's rank ends before these columns
        for (int i = q * SH_THREADS + tid; i < count * (RC / 4); i += cl * SH_THREADS) {
            const int row = i / (RC / 4), col = r0 + i % (RC / 4) * 4;
            if (col < p.r)
                *reinterpret_cast<float4*>(p.T + static_cast<int64_t>(start + row) * p.r + col) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        return;
    }

    shrink_part<BF, RC, SH_THREADS>(p, t, r0, live, q, cl, sm);
    __syncthreads();
    const float4* part4 = reinterpret_cast<const float4*>(sm);
    cluster_sync();
    const float scale = p.scales != nullptr ? p.scales[t.a] : 1.f;
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
        if (r0 + col < p.r) *reinterpret_cast<float4*>(p.T + static_cast<int64_t>(start + row) * p.r + r0 + col) = v;
    }
    cluster_sync();   // the partial sums stay until every CTA has read them
}

// ---------------------------------------------------------------------- expand
constexpr uint64_t EX_LIMIT_NS = 2000000000ull;   // of a wait

struct ExpandArgs {
    const float* T;
    const uint16_t* B;
    const int32_t *order, *tiles, *ranks;
    const void* base;
    void* Y;
    int64_t ldb, ldy;
    int M, N, n, r, ntiles;
    bool wide;           // k_lora_expand: rows of an fp32 Y start on 32-byte boundaries
    int blocks, depth;   // k_lora_expand: column blocks of a CTA, blocks of base rows in shared memory
};

// What a CTA of the kernels below works on; a bad tile has no tokens
struct Tile {
    int a, start, count, live;
};

__device__ __forceinline__ Tile entry_of(const ExpandArgs& p, int i) {   // without the rank
    Tile t;
    t.a = p.tiles[3 * i];
    t.start = p.tiles[3 * i + 1];
    t.count = p.tiles[3 * i + 2];
    if (t.count <= 0 || t.count > LR_TILE || t.start < 0 || t.start > p.M - t.count || t.a >= p.n) t.count = 0;
    t.live = 0;
    return t;
}

__device__ __forceinline__ Tile tile_of(const ExpandArgs& p, int i) {
    Tile t = entry_of(p, i);
    if (t.count > 0 && t.a >= 0) t.live = p.ranks != nullptr ? min(max(p.ranks[t.a], 0), p.r) : p.r;
    return t;
}

template <int YT>
constexpr int out_bytes = YT == HQ_F32 ? 4 : 2;

__device__ __forceinline__ float2 widen16(bool bf, uint32_t w) {
    return bf ? make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u))
              : __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// v plus one half of a word of two 16-bit values, in fp32 (no widening first)
template <bool BF>
__device__ __forceinline__ float add16(uint32_t w, bool high, float v) {
    const uint16_t h = static_cast<uint16_t>(high ? w >> 16 : w);
    float r;
    if constexpr (BF)
        asm("add.rn.f32.bf16 %0, %1, %2;" : "=f"(r) : "h"(h), "f"(v));
    else
        asm("add.rn.f32.f16 %0, %1, %2;" : "=f"(r) : "h"(h), "f"(v));
    return r;
}

__device__ __forceinline__ uint32_t narrow16(bool bf, float a, float b) {
    if (bf) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Two entries that one product may take together
__device__ __forceinline__ bool linked(const Tile& t, const Tile& next) {
    return t.count == LR_TILE && next.count > 0 && next.a == t.a && next.start == t.start + LR_TILE;
}

// The tile's rows of Y are its rows of base (or zero): tokens without an adapter
template <int YT>
__device__ void copy_cols(const ExpandArgs& p, const Tile& t, int col0, int cols);

// part q of cl of all columns
template <int YT>
__device__ void copy_rows(const ExpandArgs& p, const Tile& t, int q, int cl) {
    const int eights = p.N / 8;
    const int a = part_of(eights, q, cl), b = part_of(eights, q + 1, cl);
    copy_cols<YT>(p, t, 8 * a, 8 * (b - a));
}

template <int YT>
__device__ void copy_cols(const ExpandArgs& p, const Tile& t, int col0, int cols) {
    if (p.base == p.Y) return;   // in place
    constexpr int PER = 16 / out_bytes<YT>;
    const int vecs = (min(cols, p.N - col0)) / PER;   // N is a multiple of 8
    for (int i = threadIdx.x; i < t.count * vecs; i += blockDim.x) {
        const int m = p.order[t.start + i / vecs], col = col0 + i % vecs * PER;
        if (m < 0 || m >= p.M) continue;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (p.base != nullptr)
            v = *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.base) + (m * p.ldb + col) * out_bytes<YT>);
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.Y) + (m * p.ldy + col) * out_bytes<YT>) = v;
    }
}

// Few tokens per tile (decode): bound by the latency of its chain of loads and
// by reading B once, so plain fp32 adds without staging or hand-over.  A thread
// has two neighbouring columns; t is the same for the whole CTA (a broadcast
// load); four tokens at a time share B's values in registers.
constexpr int FEW_THREADS = 128;
constexpr int FEW_COLS = 2 * FEW_THREADS;

template <bool BF, int YT>
__global__ void __launch_bounds__(FEW_THREADS) k_lora_expand_few(const ExpandArgs p) {
    const Tile t = tile_of(p, blockIdx.y);
    const int col = blockIdx.x * FEW_COLS + 2 * threadIdx.x;
    const bool on = col < p.N;
    const uint16_t* brow = p.B + (static_cast<int64_t>(t.a) * p.N + col) * p.r;
    uint4 b[2][2];   // column, eight of sixteen rank positions
    auto load_b = [&](int c) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                b[k][e] = on && c + 8 * e < t.live ? __ldg(reinterpret_cast<const uint4*>(brow + k * p.r + c + 8 * e))
                                                   : make_uint4(0u, 0u, 0u, 0u);
    };
    int m[4];
    float y[4][2];
    auto load_base = [&](int i0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = i0 + i < t.count ? p.order[t.start + i0 + i] : -1;
            if (m[i] >= p.M) m[i] = -1;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            y[i][0] = y[i][1] = 0.f;
            if (m[i] >= 0 && on && p.base != nullptr) {
                const uint8_t* s = static_cast<const uint8_t*>(p.base) + (m[i] * p.ldb + col) * out_bytes<YT>;
                const float2 v = YT == HQ_F32 ? *reinterpret_cast<const float2*>(s)
                                              : widen16(YT == HQ_BF16, *reinterpret_cast<const uint32_t*>(s));
                y[i][0] = v.x;
                y[i][1] = v.y;
            }
        }
    };
    if (t.live > 0) {
        load_base(0);
        load_b(0);
    }
    griddep_wait();   // t is complete
    if (t.live == 0) {
        copy_cols<YT>(p, t, blockIdx.x * FEW_COLS, FEW_COLS);
        return;
    }
    for (int i0 = 0; i0 < t.count; i0 += 4) {
        if (i0 > 0) load_base(i0);
        float acc[4][2] = {};
        for (int c = 0; c < t.live; c += 16) {
            if (i0 > 0 || c > 0) load_b(c);
#pragma unroll
            for (int e = 0; e < 4; ++e) {   // four rank positions
                if (c + 4 * e >= t.live) break;
                float w[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint4 q = b[k][e >> 1];
                    const float2 lo = widen16(BF, e & 1 ? q.z : q.x), hi = widen16(BF, e & 1 ? q.w : q.y);
                    w[k][0] = lo.x; w[k][1] = lo.y; w[k][2] = hi.x; w[k][3] = hi.y;
#pragma unroll
                    for (int u = 0; u < 4; ++u)   // past the adapter's rank B is not read as a number
                        if (c + 4 * e + u >= t.live) w[k][u] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i0 + i >= t.count) break;
                    const float4 v =
                        *reinterpret_cast<const float4*>(p.T + static_cast<int64_t>(t.start + i0 + i) * p.r + c + 4 * e);
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        acc[i][k] = __fmaf_rn(v.w, w[k][3], __fmaf_rn(v.z, w[k][2], __fmaf_rn(v.y, w[k][1],
                                              __fmaf_rn(v.x, w[k][0], acc[i][k]))));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (m[i] >= 0 && on) {
                const float v0 = __fadd_rn(y[i][0], acc[i][0]), v1 = __fadd_rn(y[i][1], acc[i][1]);
                uint8_t* d = static_cast<uint8_t*>(p.Y) + (m[i] * p.ldy + col) * out_bytes<YT>;
                if constexpr (YT == HQ_F32)
                    *reinterpret_cast<float2*>(d) = make_float2(v0, v1);
                else
                    *reinterpret_cast<uint32_t*>(d) = narrow16(YT == HQ_BF16, v0, v1);
            }
    }
}

// Few tokens per tile, both products in one launch: a cluster of 8 CTAs forms a
// tile's t (each a part of K, by its first 256 threads), every CTA reads the
// partial sums of all of them from their shared memory, and then each takes an
// eighth of the columns, two neighbouring ones a thread, in plain fp32.  Bound by
// the latency of its chain of loads and barriers: threads of their own load their
// columns' B and the first token's base while t is formed, those that form it
// have theirs prefetched into L2.  Ranks up to 64; t has no place in memory.
// Against the two kernels (5.9 and 9.6 us for 1 and 16 tokens) it took 5.8 and 9.4
// us, and one launch less of host time (2.5 us), which is what a step of single
// calls waits for.
template <int RC>
constexpr int few_threads = RC <= 32 ? 768 : 512;
template <int RC>
constexpr int few_ring = SH_STAGES * (LR_TILE + RC) * 256 > 4 * LR_TILE * RC * 4 ? SH_STAGES * (LR_TILE + RC) * 256
                                                                                 : 4 * LR_TILE * RC * 4;

template <bool BF, int YT, int RC>
__global__ void __launch_bounds__(few_threads<RC>) k_lora_few(const ShrinkArgs sp, const ExpandArgs p) {
    extern __shared__ __align__(128) uint8_t sm[];   // the ring, later the partial sums; t [64][RC]
    __shared__ int rows[LR_TILE];
    constexpr int THREADS = few_threads<RC>;
    float* tt = reinterpret_cast<float*>(sm + few_ring<RC>);
    const int tid = threadIdx.x, q = blockIdx.x, cl = gridDim.x;
    const int c0 = 4 * part_of(p.N / 8, q, cl), c1 = 4 * part_of(p.N / 8, q + 1, cl);   // this CTA's pairs of columns
    ShrinkTile t;
    if (!shrink_tile(sp, blockIdx.y, t) || t.live == 0) {
        copy_rows<YT>(p, tile_of(p, blockIdx.y), q, cl);
        return;   // the whole cluster leaves
    }
    if (tid < SH_THREADS) {
#pragma unroll
        for (int j = 0; j < LR_TILE / 16; ++j)
            if ((tid & 15) == 0) rows[(tid >> 4) + 16 * j] = t.m[j];
    }
    const uint16_t* bcol = p.B + static_cast<int64_t>(t.a) * p.N * p.r;
    uint4 b[2][RC / 8];   // column, eight rank positions
    auto load_b = [&](int c) {
        const uint16_t* s = bcol + static_cast<int64_t>(2 * c) * p.r;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < RC / 8; ++e)
                b[k][e] = c < c1 && 8 * e < t.live ? __ldg(reinterpret_cast<const uint4*>(s + k * p.r) + e)
                                                   : make_uint4(0u, 0u, 0u, 0u);
    };
    auto base_at = [&](int m, int c) {
        if (p.base == nullptr || m < 0 || c >= c1) return make_float2(0.f, 0.f);
        const uint8_t* s = static_cast<const uint8_t*>(p.base) + (m * p.ldb + 2 * c) * out_bytes<YT>;
        return YT == HQ_F32 ? *reinterpret_cast<const float2*>(s) : widen16(YT == HQ_BF16, *reinterpret_cast<const uint32_t*>(s));
    };
    // the threads that do not form t have the first pairs
    const int first = c0 + (tid < SH_THREADS ? tid + THREADS - SH_THREADS : tid - SH_THREADS);
    float2 ynext = make_float2(0.f, 0.f);
    if (tid < SH_THREADS) {
        shrink_part<BF, RC, THREADS>(sp, t, 0, t.live, q, cl, sm);
    } else {
        const int m0 = p.order[t.start];
        named_bar_sync(2, THREADS);   // X and A first: t waits for them
        load_b(first);
        ynext = base_at(m0 < p.M ? m0 : -1, first);
        // everything else of this CTA's B
        const int64_t bytes = static_cast<int64_t>(c1 - c0) * 4 * p.r;
        const uint8_t* s = reinterpret_cast<const uint8_t*>(bcol + static_cast<int64_t>(2 * c0) * p.r);
        for (int64_t o = static_cast<int64_t>(THREADS - SH_THREADS) * 4 * p.r + (tid - SH_THREADS) * 128; o < bytes;
             o += (THREADS - SH_THREADS) * 128)
            prefetch_l2(s + o);
    }
    cluster_sync();
    {
        const float scale = sp.scales != nullptr ? sp.scales[t.a] : 1.f;
        const float4* part4 = reinterpret_cast<const float4*>(sm);
        for (int i = tid; i < t.count * (RC / 4); i += THREADS) {
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int h = 0; h < SH_MAX_CL; h += 4) {   // four on their way before they are added
                float4 u[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) u[c] = ld_cluster_f32x4(mapa_shared(smem_u32(part4 + i), h + c));
#pragma unroll
                for (int c = 0; c < 4; ++c) v = add4(v, u[c]);
            }
            const int col = i % (RC / 4) * 4;
            v.x = col < t.live ? __fmul_rn(v.x, scale) : 0.f;
            v.y = col + 1 < t.live ? __fmul_rn(v.y, scale) : 0.f;
            v.z = col + 2 < t.live ? __fmul_rn(v.z, scale) : 0.f;
            v.w = col + 3 < t.live ? __fmul_rn(v.w, scale) : 0.f;
            reinterpret_cast<float4*>(tt)[i] = v;
        }
    }
    // this CTA has read the others' sums; they may leave once all have (the wait is at the end)
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    __syncthreads();   // t is there
    if (tid < SH_THREADS) {
        load_b(first);
        ynext = base_at(rows[0], first);
    }
    for (int c = first; c < c1; c += THREADS) {
        if (c != first) {
            load_b(c);
            ynext = base_at(rows[0], c);
        }
        for (int i = 0; i < t.count; ++i) {
            const int m = rows[i];
            const float2 y = ynext;
            if (i + 1 < t.count) ynext = base_at(rows[i + 1], c);
            if (m < 0) continue;
            float acc[2] = {0.f, 0.f};
#pragma unroll
            for (int e = 0; e < RC / 8; ++e) {
                if (8 * e >= t.live) break;
                const float4 v0 = *reinterpret_cast<const float4*>(tt + i * RC + 8 * e);
                const float4 v1 = *reinterpret_cast<const float4*>(tt + i * RC + 8 * e + 4);
                const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    uint32_t x[4] = {b[k][e].x, b[k][e].y, b[k][e].z, b[k][e].w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        asm volatile("" : "+r"(x[u]));   // widened per token: kept widened, B would not fit the registers
                        const float2 f = widen16(BF, x[u]);
                        // past the adapter's rank B is not read as a number
                        acc[k] = __fmaf_rn(v[2 * u], 8 * e + 2 * u < t.live ? f.x : 0.f, acc[k]);
                        acc[k] = __fmaf_rn(v[2 * u + 1], 8 * e + 2 * u + 1 < t.live ? f.y : 0.f, acc[k]);
                    }
                }
            }
            uint8_t* d = static_cast<uint8_t*>(p.Y) + (m * p.ldy + 2 * c) * out_bytes<YT>;
            const float r0 = __fadd_rn(y.x, acc[0]), r1 = __fadd_rn(y.y, acc[1]);
            if constexpr (YT == HQ_F32)
                *reinterpret_cast<float2*>(d) = make_float2(r0, r1);
            else
                *reinterpret_cast<uint32_t*>(d) = narrow16(YT == HQ_BF16, r0, r1);
        }
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Whole tiles (prompts): t of two tiles (128 tokens) and blocks of 64 rows of B
// are operands of tcgen05.mma (kind::f16, 128 x 64, fp32 accumulators in tensor
// memory), so that the warps are left with what HBM sees: base in, Y out.
//  * t enters as 16-bit terms: with bf16 B two bf16 terms for a 16-bit Y (2^-18
//    of t, far below Y's rounding) and three for an fp32 Y (all of t's 24 bits); with
//    fp16 B two fp16 terms (2^-22, four times fp32's half step, for an fp32 Y too: a
//    third would be half as many products again) of the row scaled by a power of two
//    to below 2^14.
//  * operands are K-major rows of 128 bytes (64 rank positions) in the 128-byte
//    swizzle; rows of B are staged in the order that makes MMA column 8 i +
//    2 t + e of each 32 the output column 8 t + 2 i + e: a lane of the
//    16x256b accumulator layout then holds 8 consecutive outputs of a row.
//  * the next two blocks' B and the next `depth` blocks' base rows (in slots
//    that only their warp uses) are on their way (cp.async) while a block is
//    multiplied and stored; two CTAs per SM cover each other's waits.
// Two neighbouring tiles of one adapter are taken together.  What bounds it now is
// the latency of a block's chain (copies awaited, barrier, accumulators read, four
// 16-byte stores of eight rows each, copies asked for: about 2000 cycles) at two
// CTAs per SM; a third fewer instructions changed nothing.
// A ninth warp issues the products and waits for them: one thread that issues
// between its own stores held up the other warps (1300 of 3600 cycles a block).
constexpr int EX_THREADS = 256;                 // those that copy and store
constexpr int EX_ROWS = 2 * LR_TILE;            // tokens of a product
constexpr int EX_NB = 64;                       // columns of a block
constexpr int kTwoDynSmem = 228 * 1024 / 2 - 1024 - 256;   // for two CTAs on an SM, beside the static part

__host__ __device__ constexpr int ex_terms(bool bf, int yt) { return bf && yt == HQ_F32 ? 3 : 2; }
// bytes of shared memory: t, two blocks of B, base (`depth` blocks), row scales
__host__ __device__ constexpr int ex_smem(bool bf, int yt, int atoms, int depth) {
    return 1024 + ex_terms(bf, yt) * atoms * EX_ROWS * 128 + 2 * atoms * EX_NB * 128 +
           depth * EX_ROWS * EX_NB * (yt == HQ_F32 ? 4 : 2) + EX_ROWS * 4;
}

// D[tmem] (+)= A[smem] B[smem]^T, 16-bit floats, fp32 accumulators, one CTA
__device__ __forceinline__ void mma_f16_ss(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// One thread of a converged warp
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

// RK: rank up to 16, 32, 64 (one row of 128 bytes of B and t) or above (64 rank
// positions per atom, several atoms)
template <bool BF, int YT, int RK>
__global__ void __launch_bounds__(EX_THREADS + 32, 2) k_lora_expand(const ExpandArgs p) {
    constexpr int SH = RK == 16 ? 1 : RK == 32 ? 2 : 3;   // log2 of the chunks per row of B that a pass of the threads takes
    constexpr int TT = ex_terms(BF, YT);
    constexpr int ES = out_bytes<YT>;
    constexpr int PIECES = YT == HQ_F32 ? 2 : 1;
    constexpr int BASE = EX_THREADS * 4 * 16 * PIECES;   // base slots of a block
    constexpr int TATOM = EX_ROWS * 128, BATOM = EX_NB * 128;
    constexpr uint32_t IDESC = (1u << 4) | ((BF ? 1u : 0u) << 7) | ((BF ? 1u : 0u) << 10) |
                               (static_cast<uint32_t>(EX_NB >> 3) << 17) | (static_cast<uint32_t>(EX_ROWS >> 4) << 24);
    extern __shared__ uint8_t dyn[];
    __shared__ uint64_t bar_mem;
    __shared__ uint32_t tmem_mem;
    __shared__ int run_mem[2][EX_THREADS / 32 + 1];
    uint8_t* sm = dyn + ((1024u - (smem_u32(dyn) & 1023u)) & 1023u);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const bool mma_warp = warp == EX_THREADS / 32;
    const int quarter = warp & 3, c0 = 32 * (warp >> 2);   // rows 32 quarter .., columns c0 .. c0 + 31 of a block
    const int blk0 = blockIdx.x * p.blocks, blk1 = min(blk0 + p.blocks, (p.N + EX_NB - 1) / EX_NB);
    const int atoms = RK <= 64 ? 1 : (p.r + 63) / 64;
    uint8_t* tbuf = sm;
    uint8_t* bbuf = tbuf + TT * atoms * TATOM;
    uint8_t* slots = bbuf + 2 * atoms * BATOM;
    float* unscale = reinterpret_cast<float*>(slots + p.depth * BASE);
    const uint32_t bar = smem_u32(&bar_mem);
    // In a run of linked tiles (an adapter's, in a plan as hq_lora_plan makes it) the 2 k-th
    // takes the 2 k + 1-st along.  Every tile finds where its run begins: the last
    // place up to its own without a link to the one before (tile 0 has none).
    const int ti = blockIdx.y;
    auto begins = [&](int i) { return i >= 0 && (i == 0 || !linked(entry_of(p, i - 1), entry_of(p, i))); };
    const Tile next = entry_of(p, min(ti + 1, p.ntiles - 1));
    bool here = begins(ti - tid);   // asked for with the tile itself
    const Tile t = tile_of(p, ti);
    if (t.live == 0) {   // the same for the whole CTA
        griddep_wait();
        copy_cols<YT>(p, t, blk0 * EX_NB, (blk1 - blk0) * EX_NB);
        return;
    }
    constexpr int WARPS = EX_THREADS / 32 + 1;
    int first;
    for (int i = ti - tid, par = 0;; par ^= 1) {
        const unsigned w = __ballot_sync(0xFFFFFFFFu, here);
        if (lane == 0) run_mem[par][warp] = w != 0 ? i - (__ffs(w) - 1) : -1;
        __syncthreads();
        first = __reduce_max_sync(0xFFFFFFFFu, lane < WARPS ? run_mem[par][lane] : -1);
        if (first >= 0) break;
        i -= 32 * WARPS;
        here = begins(i);
    }
    if ((ti - first) & 1) {
        griddep_wait();
        return;
    }
    const int rows = t.count + (linked(t, next) ? next.count : 0);   // the last tile is not linked to itself
    if (mma_warp) {
        tmem_alloc(smem_u32(&tmem_mem), 2 * EX_NB);
        tmem_relinquish();
    }
    if (tid == 0) {
        mbar_init(bar, 1);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_mem;

    // Row l of a block of B goes to row (l & ~31) + f(l & 31) of the operand, f(l) =
    // 4 (l & 6) + 2 (l / 8) + (l & 1).  This thread's chunk of rows l0, l0 + LS, ...
    constexpr int LS = EX_THREADS >> SH < EX_NB ? EX_THREADS >> SH : EX_NB, LN = EX_NB / LS;
    const int chunk = tid & ((1 << SH) - 1), l0 = tid >> SH;
    auto b_row = [](int l) { return (l & ~31) + ((l & 6) << 2) + (((l & 31) >> 3) << 1) + (l & 1); };
    uint32_t boff[LN];
#pragma unroll
    for (int k = 0; k < LN; ++k) {
        const int row = b_row(l0 + LS * k);
        boff[k] = row * 128 + ((chunk ^ (row & 7)) << 4);
    }

    const int steps = (t.live + 15) / 16;   // k16 steps
    if (mma_warp) {
        // the product of block blk: t and B of shared memory into half blk & 1 of the accumulators
        const uint64_t td = sw128_kmajor_desc(smem_u32(tbuf)), bd = sw128_kmajor_desc(smem_u32(bbuf));
        griddep_wait();
        uint32_t phase = 0;
        bool lost = false;   // a wait gave up
        for (int blk = blk0; blk <= blk1; ++blk) {
            tc_fence_before();
            lost = __syncthreads_or(lost);   // B of this block is there, the block before it is in the accumulators
            if (lost || blk == blk1) break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t d = tm + (blk & 1) * EX_NB;
                const uint64_t b = bd + static_cast<uint32_t>((blk & 1) * atoms * (BATOM >> 4));
#pragma unroll
                for (int e = TT - 1; e >= 0; --e) {   // small terms first
                    if constexpr (RK <= 64) {
#pragma unroll
                        for (int s = 0; s < RK / 16; ++s)
                            if (s < steps)
                                mma_f16_ss(d, td + static_cast<uint32_t>(e * (TATOM >> 4) + 2 * s), b + 2u * s, IDESC,
                                           e < TT - 1 || s > 0);
                    } else {
                        for (int s = 0; s < steps; ++s)
                            mma_f16_ss(d, td + static_cast<uint32_t>((e * atoms + (s >> 2)) * (TATOM >> 4) + 2 * (s & 3)),
                                       b + static_cast<uint32_t>((s >> 2) * (BATOM >> 4) + 2 * (s & 3)), IDESC,
                                       e < TT - 1 || s > 0);
                    }
                }
                tc_commit(bar);
            }
            __syncwarp();
            lost = !mbar_wait(bar, phase, EX_LIMIT_NS);
            phase ^= 1u;
        }
        __syncthreads();
        tmem_dealloc(tm, 2 * EX_NB);
        return;
    }
    int m[2][2];                            // this lane's rows 32 quarter + 16 f + 8 h + g
    const uint8_t* ysrc[2][2];
    uint8_t* ydst[2][2];
#pragma unroll
    for (int f = 0; f < 2; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = 32 * quarter + 16 * f + 8 * h + g;
            m[f][h] = i < rows ? p.order[t.start + i] : -1;
            if (m[f][h] >= p.M) m[f][h] = -1;
            const int64_t col = static_cast<int64_t>(blk0) * EX_NB + c0 + 8 * t4;
            const int64_t row = max(m[f][h], 0);
            ysrc[f][h] = p.base != nullptr && m[f][h] >= 0
                             ? static_cast<const uint8_t*>(p.base) + (row * p.ldb + col) * ES
                             : nullptr;
            ydst[f][h] = static_cast<uint8_t*>(p.Y) + (row * p.ldy + col) * ES;
        }
    // the next block to copy, of B and of base: pointers that move on block by block
    const uint16_t* bsrc =
        p.B + (static_cast<int64_t>(t.a) * p.N + static_cast<int64_t>(blk0) * EX_NB + l0) * p.r + 8 * chunk;
    int bleft = l0 < EX_NB ? p.N - blk0 * EX_NB - l0 : 0;   // this thread's rows in bounds: LS k < bleft
    int bblk = blk0;
    auto load_b = [&]() {
        if (bblk < blk1) {
            const uint32_t bd = smem_u32(bbuf) + (bblk & 1) * atoms * BATOM;
#pragma unroll 1
            for (int at = 0; at < atoms; ++at) {
                const int j = 64 * at + 8 * chunk;   // rank position of the chunk
                if (j < 16 * steps && l0 < EX_NB) {
                    const uint16_t* src = bsrc + 64 * at;
#pragma unroll
                    for (int k = 0; k < LN; ++k) {
                        if (j < t.live && LS * k < bleft)
                            cp_async16(bd + at * BATOM + boff[k], src);
                        else
                            cp_async16_z(bd + at * BATOM + boff[k], p.B, 0);
                        src += static_cast<int64_t>(LS) * p.r;
                    }
                }
            }
            bsrc += static_cast<int64_t>(EX_NB) * p.r;
            bleft -= EX_NB;
            ++bblk;
        }
    };
    // the last chunk of an adapter whose rank is no multiple of 8: what lies behind
    // the rank is not read as a number (each thread mends what it copied)
    auto mend = [&](int blk) {
        const int j0 = t.live & ~7;
        if ((t.live & 7) == 0 || chunk != ((j0 & 63) >> 3) || l0 >= EX_NB) return;
        uint8_t* bd = bbuf + ((blk & 1) * atoms + (j0 >> 6)) * BATOM;
#pragma unroll
        for (int k = 0; k < LN; ++k) {
            uint16_t* d = reinterpret_cast<uint16_t*>(bd + boff[k]);
            for (int e = t.live & 7; e < 8; ++e) d[e] = 0;
        }
    };
    const uint32_t slot0 = smem_u32(slots) + tid * 16;
    int yleft = p.N - blk0 * EX_NB - c0 - 8 * t4;   // columns left for this lane
    int64_t ybytes = 0;                              // from the first block on
    // a warp whose rows are all there, with a base: no checks but for the last block
    const bool whole = __all_sync(0xFFFFFFFFu, p.base != nullptr && m[0][0] >= 0 && m[0][1] >= 0 && m[1][0] >= 0 && m[1][1] >= 0);
    // Chunk j (16 bytes) of the 8 that four lanes share of an fp32 row is asked for by
    // lane (j ^ j / 4) % 4, so that each of its two copies takes whole sectors with
    // its neighbours' (half sectors took 27% longer at 8192 x 11008, rank 32), and its reads
    // have no bank conflicts.  ahead(e): where
    // copy e lies, in chunks from this lane's first column
    auto ahead = [&](int e) { return PIECES == 1 ? 0 : 4 * e + (t4 ^ e) - 2 * t4; };
    auto base_slot = [&](int e) {   // of this lane's chunk e
        return PIECES == 1 ? 0 : (t4 >> 1) * EX_THREADS * 16 + 16 * ((((2 * t4 + e) & 3) ^ (t4 >> 1)) - t4);
    };
    auto load_base = [&](bool more, int slot) {
        if (!more) return;
        const uint32_t sd = slot0 + slot * BASE;
        const bool all = whole && yleft >= 64;
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (all || ysrc[f][h] != nullptr) {
#pragma unroll
                    for (int e = 0; e < PIECES; ++e)
                        if (all || yleft > (16 / ES) * ahead(e))
                            cp_async16(sd + ((f * 2 + h) * PIECES + e) * EX_THREADS * 16, ysrc[f][h] + ybytes + 16 * ahead(e));
                }
            }
        ybytes += EX_NB * ES;
        yleft -= EX_NB;
    };
    load_b();
    load_base(true, 0);
    cp_async_commit();
    load_b();
    cp_async_commit();
    for (int k = 1; k < p.depth; ++k) load_base(blk0 + k < blk1, k);
    cp_async_commit();
    griddep_wait();   // t is complete
    {   // t in 16-bit terms: two threads per row take alternate chunks of 8 positions
        const int row = tid >> 1;
        const float* src = p.T + static_cast<int64_t>(t.start + row) * p.r;
        float scale = 1.f;
        if constexpr (!BF) {
            float top = 0.f;
            if (row < rows)
                for (int c = tid & 1; 8 * c < t.live; c += 2)
#pragma unroll
                    for (int e = 0; e < 8; e += 4) {
                        const float4 v = *reinterpret_cast<const float4*>(src + 8 * c + e);
                        top = fmaxf(top, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
                    }
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            // 2^(13 - e) for top in [2^e, 2^(e+1)); e >= -100 keeps it finite
            const int e = max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100);
            if (top > 0.f && top < INFINITY) scale = __uint_as_float(static_cast<uint32_t>(127 + 13 - e) << 23);
            if ((tid & 1) == 0) unscale[row] = __fdiv_rn(1.f, scale);   // a power of two: exact
        }
        if (row < rows)
            for (int c = tid & 1; c < 2 * steps; c += 2) {
                float v[8] = {};
                if (8 * c < p.r) {
                    const float4 a = *reinterpret_cast<const float4*>(src + 8 * c);
                    const float4 b = *reinterpret_cast<const float4*>(src + 8 * c + 4);
                    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
                    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
                }
                if constexpr (!BF) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[k] = __fmul_rn(v[k], scale);
                }
#pragma unroll
                for (int e = 0; e < TT; ++e) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        w[k] = narrow16(BF, v[2 * k], v[2 * k + 1]);
                        const float2 f = widen16(BF, w[k]);
                        // the rest; none where the term is not finite
                        v[2 * k] = fabsf(f.x) < INFINITY ? __fsub_rn(v[2 * k], f.x) : 0.f;
                        v[2 * k + 1] = fabsf(f.y) < INFINITY ? __fsub_rn(v[2 * k + 1], f.y) : 0.f;
                    }
                    *reinterpret_cast<uint4*>(tbuf + (e * atoms + (c >> 3)) * TATOM + row * 128 +
                                              (((c & 7) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
    }
    // Block b + 1 is multiplied while block b is stored.  Copy groups in order: B of
    // b + 2 (over the B just multiplied), then the base rows of b + depth (over
    // those just used); the product of b + 1 needs all but the last of them.
    cp_async_wait_group<2>();
    mend(blk0);
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads_or(0);
    float us[2][2] = {{1.f, 1.f}, {1.f, 1.f}};
    if constexpr (!BF) {
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int h = 0; h < 2; ++h) us[f][h] = unscale[32 * quarter + 16 * f + 8 * h + g];
    }
    int left = p.N - blk0 * EX_NB - c0 - 8 * t4;
    int64_t dbytes = 0;
    int slot = 0;
    for (int blk = blk0; blk < blk1; ++blk) {
        if (p.depth > 1 || blk == blk0)
            cp_async_wait_group<1>();
        else
            cp_async_wait_all();
        if (blk + 1 < blk1) {
            mend(blk + 1);
            fence_proxy_async_smem();
        }
        tc_fence_before();
        if (__syncthreads_or(0)) break;   // the product of this block is done (or was given up)
        load_b();
        cp_async_commit();
        if (32 * quarter < rows) {
            tc_fence_after();
            const uint8_t* sd = slots + slot * BASE + tid * 16;
            uint32_t acc[2][16];
            const uint32_t at = tm + (static_cast<uint32_t>(32 * quarter) << 16) + (blk & 1) * EX_NB + c0;
            tmem_ld_16x256b_x4(at, acc[0]);
            tmem_ld_16x256b_x4(at + (16u << 16), acc[1]);
            tmem_wait_ld();
            auto store = [&](auto checked) {
                constexpr bool CHECK = decltype(checked)::value;
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        if (CHECK && (m[f][h] < 0 || left <= 0)) continue;
                        uint32_t both[PIECES][4];
#pragma unroll
                        for (int e = 0; e < PIECES; ++e) {
                            uint4 y = make_uint4(0u, 0u, 0u, 0u);
                            if (!CHECK || p.base != nullptr)
                                y = *reinterpret_cast<const uint4*>(sd + (f * 2 + h) * PIECES * EX_THREADS * 16 + base_slot(e));
                            uint32_t w[4] = {y.x, y.y, y.z, y.w};
                            constexpr int PER = YT == HQ_F32 ? 1 : 2;   // outputs per word
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const int o = (4 * e + k) * PER;   // output 2 i + c (of 8) is acc[4 i + 2 h + c]
                                float v0 = __uint_as_float(acc[f][4 * (o / 2) + 2 * h + (o & 1)]);
                                if constexpr (!BF) v0 = __fmul_rn(v0, us[f][h]);
                                if constexpr (YT == HQ_F32) {
                                    w[k] = __float_as_uint(__fadd_rn(__uint_as_float(w[k]), v0));
                                } else {
                                    float v1 = __uint_as_float(acc[f][4 * (o / 2) + 2 * h + 1]);
                                    if constexpr (!BF) v1 = __fmul_rn(v1, us[f][h]);
                                    w[k] = narrow16(YT == HQ_BF16, add16<YT == HQ_BF16>(w[k], false, v0),
                                                    add16<YT == HQ_BF16>(w[k], true, v1));
                                }
                            }
                            if (PIECES == 1 || !p.wide)
                                reinterpret_cast<uint4*>(ydst[f][h] + dbytes)[e] = make_uint4(w[0], w[1], w[2], w[3]);
#pragma unroll
                            for (int k = 0; k < 4; ++k) both[e][k] = w[k];
                        }
                        if constexpr (PIECES == 2) {
                            // the halves of a sector one by one took 12% longer (8192 x 11008, rank 32)
                            if (p.wide)
                                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                                                 ydst[f][h] + dbytes),
                                             "r"(both[0][0]), "r"(both[0][1]), "r"(both[0][2]), "r"(both[0][3]),
                                             "r"(both[1][0]), "r"(both[1][1]), "r"(both[1][2]), "r"(both[1][3])
                                             : "memory");
                        }
                    }
            };
            if (whole && __all_sync(0xFFFFFFFFu, left > 0))
                store(std::false_type{});
            else
                store(std::true_type{});
            if constexpr (PIECES == 2) __syncwarp();   // the slots are the warp's
            load_base(blk + p.depth < blk1, slot);
        }
        cp_async_commit();
        slot = slot + 1 == p.depth ? 0 : slot + 1;
        left -= EX_NB;
        dbytes += EX_NB * ES;
    }
    cp_async_wait_all();
    tc_fence_before();
    __syncthreads();   // the accumulators may go
}

bool lr_al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <bool BF, int RC>
hq_status launch_shrink(const ShrinkArgs& a, int tiles, cudaStream_t st) {
    constexpr int ring = SH_STAGES * (LR_TILE + RC) * 256, part = 4 * LR_TILE * RC * 4;
    constexpr int smem = ring > part ? ring : part;
    auto kern = k_lora_shrink<BF, RC>;
    static SmemOptIn opt_in;
    if (!allow_smem(opt_in, kern, smem)) return HQ_ERR_CUDA;
    // K is cut as far as the GPU holds all CTAs at once
    const int z = (a.r + RC - 1) / RC, slots = 148 * sh_ctas<RC>;
    int cl = SH_MAX_CL;
    while (cl > 1 && static_cast<int64_t>(tiles) * z * cl > slots) cl /= 2;
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

template <bool BF, int YT>
hq_status launch_expand(ExpandArgs a, int tiles, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.stream = st;
    // may start while k_lora_shrink runs; it waits for that grid's completion
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int atoms = (a.r + 63) / 64;
    // few tokens for each possible tile (see launch_lora_y), or (bf16 with fp32 Y above rank
    // 192) too much for shared memory: 2048 x 4096 -> 4096, rank 256 takes 787 us so
    if (a.M < 16 * tiles || ex_smem(BF, YT, atoms, 1) > kMaxDynSmem) {
        cfg.gridDim = dim3((a.N + FEW_COLS - 1) / FEW_COLS, tiles);
        cfg.blockDim = dim3(FEW_THREADS);
        return cudaLaunchKernelEx(&cfg, k_lora_expand_few<BF, YT>, a) == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
    }
    // a CTA stages its tiles' t once for all its blocks of columns: as many CTAs as
    // the GPU holds at once (two per SM), counting at most `heads` tiles that lead
    // a pair; three rounds of smaller CTAs measured 2% (8192 x 28672) to 15%
    // (2048 x 4096) slower
    const int64_t nblk = (a.N + EX_NB - 1) / EX_NB;
    const int heads = (tiles + (a.n < tiles ? a.n : tiles) + 1) / 2;
    auto strips_for = [&](int per_sm) {
        const int64_t s = 148 * per_sm / heads;
        return s < 1 ? 1 : s > nblk ? nblk : s;
    };
    int64_t strips = strips_for(2);
    a.wide = YT == HQ_F32 && (reinterpret_cast<uintptr_t>(a.Y) & 31u) == 0 && a.ldy % 8 == 0;
    a.depth = 3;
    // Where every SM is sure to have a CTA, two of them per SM are worth more than blocks
    // asked for ahead (fp32 Y, 8192 x 4096 -> 11008, rank 32: fp16 173 us in place of 185,
    // but bf16 166 of 162; 2024 x 168 -> 1320: 17.1, 19.2), and where shared memory has
    // room for one only (ranks above 64), one round of larger CTAs more than two of smaller
    // ones (2048 x 4096 -> 4096, rank 128: 45 us, 48.7, but with fp32 Y 67.5 of 66; 8192 x
    // 4096 -> 11008, rank 256: 207, 219).  With fewer CTAs it is the other way round (442
    // tokens of one adapter, 184 -> 3864, fp32 Y: 22 in place of 16 us).  All as measured when
    // it was tried; the same cases take 163, 166, 16.6, 45, 53, 208 and 14.2 us now.
    if ((static_cast<int64_t>(a.M) + EX_ROWS - 1) / EX_ROWS * strips >= 148) {
        while (a.depth > 1 && ex_smem(BF, YT, atoms, a.depth) > kTwoDynSmem) --a.depth;
        if (ex_smem(BF, YT, atoms, a.depth) > kTwoDynSmem) {
            a.depth = 3;
            strips = strips_for(1);
        }
    }
    while (a.depth > 1 && ex_smem(BF, YT, atoms, a.depth) > kMaxDynSmem) --a.depth;
    const int smem = ex_smem(BF, YT, atoms, a.depth);
    const int rk = a.r <= 16 ? 0 : a.r <= 32 ? 1 : a.r <= 64 ? 2 : 3;
    auto kern = rk == 0   ? k_lora_expand<BF, YT, 16>
                : rk == 1 ? k_lora_expand<BF, YT, 32>
                : rk == 2 ? k_lora_expand<BF, YT, 64>
                          : k_lora_expand<BF, YT, 256>;
    static SmemOptIn opt_in[4];
    if (!allow_smem(opt_in[rk], kern, smem)) return HQ_ERR_CUDA;
    const int64_t per = (nblk + strips - 1) / strips;
    a.blocks = static_cast<int>(per);
    a.ntiles = tiles;
    cfg.gridDim = dim3(static_cast<unsigned>((nblk + per - 1) / per), tiles);
    cfg.blockDim = dim3(EX_THREADS + 32);
    cfg.dynamicSmemBytes = smem;
    return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

template <bool BF, int YT, int RC>
hq_status launch_few(const ShrinkArgs& s, const ExpandArgs& e, int tiles, cudaStream_t st) {
    constexpr int smem = few_ring<RC> + LR_TILE * RC * 4;
    auto kern = k_lora_few<BF, YT, RC>;
    static SmemOptIn opt_in;
    if (!allow_smem(opt_in, kern, smem)) return HQ_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(SH_MAX_CL, tiles);
    cfg.blockDim = dim3(few_threads<RC>);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = SH_MAX_CL;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, s, e) == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

template <bool BF, int YT>
hq_status launch_lora_y(const ShrinkArgs& s, const ExpandArgs& e, int tiles, cudaStream_t st) {
    // How many tokens a tile holds is known on the GPU only; `tiles` is the plan's bound
    // M / 64 + min(n + 1, M), which grows with the adapters in memory.  Below 16 tokens for
    // each of them the few-token form: what decode wants (1 and 16 tokens 5.8 and 9.4 us in
    // place of 5.9 and 9.6 for two kernels), but also what long prompts get beside many
    // resident adapters: 1024 tokens of one request, 4096 -> 11008, rank 32, take 26 us
    // beside 8 adapters and 156 beside 64, 4096 tokens of 12 requests 60 beside 16 and 405
    // beside 256.
    if (s.M < 16 * tiles && s.r <= 64)
        return s.r <= 16   ? launch_few<BF, YT, 16>(s, e, tiles, st)
               : s.r <= 32 ? launch_few<BF, YT, 32>(s, e, tiles, st)
                           : launch_few<BF, YT, 64>(s, e, tiles, st);
    const hq_status r = s.r <= 16 ? launch_shrink<BF, 16>(s, tiles, st)
                        : s.r <= 32 ? launch_shrink<BF, 32>(s, tiles, st)
                                    : launch_shrink<BF, 64>(s, tiles, st);
    return r != HQ_OK ? r : launch_expand<BF, YT>(e, tiles, st);
}

template <bool BF>
hq_status launch_lora(const ShrinkArgs& s, const ExpandArgs& e, int yt, int tiles, cudaStream_t st) {
    if (yt == HQ_F16) return launch_lora_y<BF, HQ_F16>(s, e, tiles, st);
    if (yt == HQ_BF16) return launch_lora_y<BF, HQ_BF16>(s, e, tiles, st);
    return launch_lora_y<BF, HQ_F32>(s, e, tiles, st);
}

}  // namespace
}  // namespace hq

using namespace hq;

extern "C" int64_t hq_lora_max_tiles(int64_t M, int64_t n) {
    if (M <= 0 || n < 0) return 0;
    return M / LR_TILE + (n < M ? n + 1 : M);
}

extern "C" hq_status hq_lora_plan(const int32_t* ids, int64_t M, int64_t n, int32_t* order, int32_t* tiles,
                                  void* stream) {
    if (M < 0 || n < 0) return HQ_ERR_ARG;
    if (n > LR_MAX_ADAPTERS || hq_lora_max_tiles(M, n) > 65535) return HQ_ERR_UNSUPPORTED;
    if (M == 0) return HQ_OK;
    if (!ids || !order || !tiles || ids == order || ids == tiles || order == tiles) return HQ_ERR_ARG;
    int cl = 1;
    while (cl < PL_MAX_CL && M > static_cast<int64_t>(PL_RUN) * cl) cl *= 2;
    // a warp per 32 tokens, up to a full CTA
    const int nb = static_cast<int>(n) + 1;
    const int64_t per = (M + cl - 1) / cl;
    const int W = static_cast<int>(per < PL_THREADS ? (per + 31) / 32 : PL_THREADS / 32);
    const int run = static_cast<int>(((per + W - 1) / W + 31) / 32 * 32);
    const int smem = (W * nb + 2 * (nb + 1) + nb) * 4;
    // a thread per bucket and one for the totals
    const int threads = 32 * W > nb + 1 ? 32 * W : (nb + 1 + 31) / 32 * 32;
    static SmemOptIn opt_in;
    if (!allow_smem(opt_in, k_lora_plan, smem)) return HQ_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cl);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cl;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cl > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_lora_plan, ids, static_cast<int>(M), static_cast<int>(n), W, run, order,
                                             tiles, static_cast<int>(hq_lora_max_tiles(M, n)));
    return e == cudaSuccess ? HQ_OK : HQ_ERR_CUDA;
}

extern "C" size_t hq_lora_workspace_size(int64_t M, int32_t r_max) {
    if (M <= 0 || r_max <= 0) return 0;
    const size_t row = static_cast<size_t>(r_max) * sizeof(float);
    return static_cast<size_t>(M) > SIZE_MAX / row ? SIZE_MAX : M * row;
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
    if (X == Y && ld_x * 2 != ld_y * es) return HQ_ERR_ARG;   // rows of Y over other rows of X
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
