// Low-rank adapters of many requests beside the FP8 projection:
//
//   y[t][c] = bf16( sum_g a_s[t][g] w_s[c/128][g] P_g[t][c] + sum_r v[t][r] B_a[c][r] ),
//   v[t][r] = scaling[a] * sum_k x[t][k] A_a[r][k],     a = ids[t]
//
// The kernels here read x once: they quantize it for the projection, exactly
// as the activation quantizer does, and form v (products of bf16 values, sums
// in fp32). The projection's kernels (gemm.cu) then add the second sum to
// their fp32 accumulators, so the output is rounded once and no pass over y
// is needed. v is fp32 for the decode kernel, which serves large decode batches
// with many adapters too, 64 rows at a time. The pair kernel multiplies on the
// tensor cores, whose operand type is bf16: there v is the sum of two bf16 parts,
// hi = bf16(v) and lo = bf16(v - hi) (v - hi is exact in fp32), and both are
// multiplied with B into the same fp32 sum. hi + lo is off by at most 2^-8 of lo,
// 2^-16 |v|: no more than what summing K >= 128 products in fp32 may be off by
// ((K + 2) 2^-23 of their magnitudes). One part alone, 2^-8 |v|, reached the
// outputs where the terms of the second sum cancel: up to ten times the bound
// (257 rows, K = 256, rank 8).
//
// Up to 64 rows (a decode batch, each row with an adapter of its own), unless K is
// so long that a row does not fit in shared memory: a cluster per row, its CTAs splitting K; bound by reading every used A once.
// More rows: 64 rows and a part of K per CTA, on the legacy tensor path
// (mma.sync): 2 M rank K flops are a hundredth of the projection's, and what
// binds is the latency of bringing x and A through L2. Other CTAs of the same
// launch quantize meanwhile; doing both in one CTA took 50 us at 4576 rows,
// K = 6144, rank 64, three times what either needs.
#include <cuda_bf16.h>

#include <mutex>

#include "group_quant.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "ptx_routed.cuh"
#include "routed.h"
#include "team_quant.cuh"

namespace fp8q {

namespace {

struct PrepShape {
    uint32_t m, n, k, mp, adapters, rank;
    uint32_t passes;  // many rows: clusters per 64 rows
    uint32_t v_fp32;
};

// ------------------------------------------------------- decode widths --

constexpr uint32_t kRowThreads = 128;
constexpr uint32_t kRowMaxSplit = 8;
constexpr uint32_t kRowsTogether = 4;  // rows of A that a warp multiplies at a time
constexpr uint32_t kPrefetchBytes = 32u << 20;  // of B in all: a part of L2 that leaves room for the weight stream
constexpr uint32_t kRowChunks = 3;     // 256-column pieces of them in flight together

// Cluster of `split` CTAs per row; CTA `rank` owns the K groups rank*G/split ..
// Everything that misses the caches is requested as soon as the row's adapter is
// known: the first rows of A before x is quantized, and the adapter's B, which
// the projection reads at its end, into L2.
__global__ void __launch_bounds__(kRowThreads)
    lora_rows_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ ids, const uint16_t* __restrict__ a_w,
                     const uint16_t* __restrict__ b_w, const float* __restrict__ scaling, uint8_t* __restrict__ q,
                     float* __restrict__ s_k, float* __restrict__ v, uint32_t split, const PrepShape sh) {
    extern __shared__ __align__(128) uint8_t smem[];
    const uint32_t G = sh.k / 128u;
    const uint32_t t = blockIdx.x / split, rank = cluster_ctarank();
    const uint32_t g0 = rank * G / split, g1 = (rank + 1) * G / split;
    const uint32_t len = (g1 - g0) * 128u;
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint16_t* xs = reinterpret_cast<uint16_t*>(smem);
    float* part = reinterpret_cast<float*>(smem + ((G + split - 1) / split) * 256u);
    grid_dependency_wait();
    trigger_dependents();
    const uint32_t a = static_cast<uint32_t>(__ldg(ids + t));
    const bool has = a < sh.adapters;
    const uint16_t* a_rows = a_w + (has ? static_cast<size_t>(a) * sh.rank * sh.k : 0u) + g0 * 128u;

    uint4 w[kRowChunks][kRowsTogether];
    auto request = [&](uint32_t r0, uint32_t c0) {
#pragma unroll
        for (uint32_t i = 0; i < kRowChunks; ++i)
#pragma unroll
            for (uint32_t j = 0; j < kRowsTogether; ++j) {
                const uint32_t c = c0 + i * 256u + lane * 8u;
                w[i][j] = has && r0 < sh.rank && c < len ? ld_stream16(a_rows + static_cast<size_t>(r0 + j) * sh.k + c) : make_uint4(0u, 0u, 0u, 0u);
            }
    };
    request(warp * kRowsTogether, 0);
    if (has) {
        const uint8_t* b = reinterpret_cast<const uint8_t*>(b_w + static_cast<size_t>(a) * sh.n * sh.rank);
        const uint64_t all = static_cast<uint64_t>(sh.n) * sh.rank * 2u;
        const uint32_t share = kPrefetchBytes / sh.m;
        const uint32_t bytes = all < share ? static_cast<uint32_t>(all) : share;
        for (uint32_t at = (rank * kRowThreads + threadIdx.x) * 128u; at < bytes; at += split * kRowThreads * 128u)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(b + at));
    }

    const uint32_t l = threadIdx.x & 7u;
    for (uint32_t gb = 0; gb < g1 - g0; gb += kRowThreads / 8u) {
        const uint32_t gl = gb + (threadIdx.x >> 3);
        const bool ok = gl < g1 - g0;
        const size_t off = static_cast<size_t>(t) * sh.k + static_cast<size_t>(g0 + (ok ? gl : 0u)) * 128u + l * 8u;
        const uint4 va = ld_stream16(x + off), vb = ld_stream16(x + off + 64);
        uint2 ca, cb;
        const float s = encode_team(va, vb, &ca, &cb);
        if (ok) {
            store_team(q + off - l * 8u, l, ca, cb);
            if (l == 0) s_k[static_cast<size_t>(g0 + gl) * sh.mp + t] = s;
            *reinterpret_cast<uint4*>(xs + gl * 128u + l * 8u) = va;
            *reinterpret_cast<uint4*>(xs + gl * 128u + 64u + l * 8u) = vb;
        }
    }
    zero_kmajor_pad(s_k, sh.m, sh.mp, G);
    __syncthreads();
    if (has) {
        for (uint32_t r0 = warp * kRowsTogether; r0 < sh.rank; r0 += kRowThreads / 32u * kRowsTogether) {
            float acc[kRowsTogether] = {};
            for (uint32_t c0 = 0; c0 < len; c0 += kRowChunks * 256u) {
                if (c0 != 0 || r0 != warp * kRowsTogether) request(r0, c0);
#pragma unroll
                for (uint32_t i = 0; i < kRowChunks; ++i) {
                    const uint32_t c = c0 + i * 256u + lane * 8u;
                    if (c >= len) break;
                    float f[8];
                    widen8(*reinterpret_cast<const uint4*>(xs + c), f);
#pragma unroll
                    for (uint32_t j = 0; j < kRowsTogether; ++j) {
                        float h[8];
                        widen8(w[i][j], h);
#pragma unroll
                        for (uint32_t e = 0; e < 8; ++e) acc[j] = fmaf(f[e], h[e], acc[j]);
                    }
                }
            }
#pragma unroll
            for (uint32_t j = 0; j < kRowsTogether; ++j) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xFFFFFFFFu, acc[j], o);
                if (lane == 0) part[r0 + j] = acc[j];
            }
        }
    }
    cluster_sync_all();
    if (has) {
        const float scale = __ldg(scaling + a);
        for (uint32_t r = rank * kRowThreads + threadIdx.x; r < sh.rank; r += split * kRowThreads) {
            float n[kRowMaxSplit], sum = 0.0f;
#pragma unroll
            for (uint32_t p = 0; p < kRowMaxSplit; ++p) {
                n[p] = 0.0f;
                if (p < split)
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(n[p]) : "r"(mapa_shared(smem_addr(part + r), p)) : "memory");
            }
#pragma unroll
            for (uint32_t p = 0; p < kRowMaxSplit; ++p) sum += n[p];
            v[static_cast<size_t>(t) * sh.rank + r] = scale * sum;
        }
    }
    cluster_sync_all();  // no CTA leaves while another reads its sums
}

// ------------------------------------------------------------ many rows --

constexpr uint32_t kTileRows = 64;
constexpr uint32_t kTileThreads = 256;
constexpr uint32_t kSlab = 64;       // columns of v per pass
constexpr uint32_t kTileStages = 2;
constexpr uint32_t kTileMaxSplit = 8;
constexpr uint32_t kPassCtas = 4;
constexpr uint32_t kRowBytes = 272;  // 128 bf16 and 16 bytes that spread rows over the banks
constexpr uint32_t kXBytes = kTileRows * kRowBytes;
constexpr uint32_t kABytes = kSlab * kRowBytes;
constexpr uint32_t kStageBytes = kXBytes + kABytes;

constexpr uint32_t kTeamGroups = 4;

// CTAs that quantize `groups` groups.
__host__ __device__ __forceinline__ uint32_t team_parts(uint32_t groups) {
    constexpr uint32_t per = kTileThreads / 8u * kTeamGroups;
    return (groups + per - 1) / per;
}

struct TileSmem {
    uint8_t stage[kTileStages][kStageBytes];
    int32_t ids[kTileRows];
    int32_t list[256];
    uint32_t listed;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(ok ? 16u : 0u) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 128 groups of x (row-major order, CTA `part`) by teams of eight lanes, all of a
// team's loads in flight together; the CTAs share the zeroing of the scales' pad.
__device__ __forceinline__ void quantize_groups(const uint16_t* __restrict__ x, uint8_t* __restrict__ q, float* __restrict__ s_k,
                                                uint32_t part, const PrepShape& sh) {
    const uint32_t G = sh.k / 128u, groups = sh.m * G, l = threadIdx.x & 7u;
    uint32_t at[kTeamGroups];
    uint4 a[kTeamGroups], b[kTeamGroups];
#pragma unroll
    for (uint32_t i = 0; i < kTeamGroups; ++i) {
        at[i] = (part * kTeamGroups + i) * (kTileThreads / 8u) + (threadIdx.x >> 3);
        const uint16_t* src = x + static_cast<size_t>(at[i] < groups ? at[i] : 0u) * 128u + l * 8u;
        a[i] = ld_stream16(src);
        b[i] = ld_stream16(src + 64);
    }
#pragma unroll
    for (uint32_t i = 0; i < kTeamGroups; ++i) {
        uint2 ca, cb;
        const float s = encode_team(a[i], b[i], &ca, &cb);
        if (at[i] < groups) {
            store_team(q + static_cast<size_t>(at[i]) * 128u, l, ca, cb);
            const uint32_t t = at[i] / G;
            if (l == 0) s_k[static_cast<size_t>(at[i] - t * G) * sh.mp + t] = s;
        }
    }
    const uint32_t pad = sh.mp - sh.m, parts = team_parts(groups);
    for (uint32_t i = part * kTileThreads + threadIdx.x; i < pad * G; i += parts * kTileThreads)
        s_k[static_cast<size_t>(i / pad) * sh.mp + sh.m + i % pad] = 0.0f;
}

// Cluster of `split` CTAs per 64 rows; CTA `rank` owns the K groups rank*G/split ..
// One pass over its part of K for each adapter among the 64 rows and each 64 of
// the rank. Every 64 rows have sh.passes clusters that take these passes in turn:
// a request boundary inside the rows does not double the time, nor do the many
// adapters of a large decode batch multiply it. The clusters after them quantize x.
// The CTAs' parts of v are added through distributed shared memory in rank order.
// For the pair kernel the first CTA of every 256 rows also lists the adapters that
// those rows use, in order of first use.
__global__ void __launch_bounds__(kTileThreads)
    lora_tiles_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ ids, const uint16_t* __restrict__ a_w,
                      const float* __restrict__ scaling, uint8_t* __restrict__ q, float* __restrict__ s_k,
                      void* __restrict__ v, int32_t* __restrict__ lists, uint32_t split, const PrepShape sh) {
    extern __shared__ __align__(128) uint8_t smem[];
    TileSmem& sm = *reinterpret_cast<TileSmem*>(smem);
    const uint32_t G = sh.k / 128u;
    const uint32_t blocks = (sh.m + kTileRows - 1) / kTileRows;
    const uint32_t cluster = blockIdx.x / split, rank = cluster_ctarank();
    const uint32_t turn = cluster / blocks;  // of the passes
    const uint32_t row0 = (cluster - turn * blocks) * kTileRows;
    const uint32_t g0 = rank * G / split, g1 = (rank + 1) * G / split;
    const uint32_t tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dependency_wait();
    trigger_dependents();
    if (turn >= sh.passes) {
        quantize_groups(x, q, s_k, (cluster - sh.passes * blocks) * split + rank, sh);
        return;
    }
    if (tid < kTileRows) {
        const int32_t id = row0 + tid < sh.m ? __ldg(ids + row0 + tid) : -1;
        sm.ids[tid] = static_cast<uint32_t>(id) < sh.adapters ? id : -1;
    }
    if (lists && turn == 0 && rank == 0 && row0 % 256u == 0) {
        // One warp after the other appends the ids that it is the first to see.
        const int32_t id = row0 + tid < sh.m ? __ldg(ids + row0 + tid) : -1;
        const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
        bool first = static_cast<uint32_t>(id) < sh.adapters && (same & ((1u << lane) - 1u)) == 0;
        if (tid == 0) sm.listed = 0;
        for (uint32_t w = 0; w < kTileThreads / 32; ++w) {
            __syncthreads();
            if (w == warp) {
                const uint32_t before = sm.listed;
                if (first)
                    for (uint32_t i = 0; i < before; ++i) first = first && sm.list[i] != id;
                const uint32_t votes = __ballot_sync(0xFFFFFFFFu, first);
                if (first) sm.list[before + __popc(votes & ((1u << lane) - 1u))] = id;
                if (lane == 0) sm.listed = before + __popc(votes);
            }
        }
        __syncthreads();
        int32_t* list = lists + static_cast<size_t>(row0 / 256u) * kAdapterList;
        if (tid < sm.listed) list[1 + tid] = sm.list[tid];
        if (tid == 0) list[0] = static_cast<int32_t>(sm.listed);
    }
    __syncthreads();
    const int32_t id0 = sm.ids[lane], id1 = sm.ids[lane + 32];
    uint64_t todo = __ballot_sync(0xFFFFFFFFu, id0 >= 0) | static_cast<uint64_t>(__ballot_sync(0xFFFFFFFFu, id1 >= 0)) << 32;
    uint32_t pass = 0;
    while (todo) {
        const int32_t a = sm.ids[__ffsll(static_cast<long long>(todo)) - 1];
        todo &= ~(__ballot_sync(0xFFFFFFFFu, id0 == a) | static_cast<uint64_t>(__ballot_sync(0xFFFFFFFFu, id1 == a)) << 32);
        for (uint32_t slab = 0; slab < sh.rank; slab += kSlab, ++pass) {
            if (pass % sh.passes != turn) continue;
            auto issue = [&](uint32_t i) {
                if (g0 + i < g1) {
                    const uint32_t base = smem_addr(sm.stage[i % kTileStages]);
                    const size_t col = static_cast<size_t>(g0 + i) * 128u;
#pragma unroll
                    for (uint32_t j = 0; j < kTileRows * 16u / kTileThreads; ++j) {
                        const uint32_t c = tid + j * kTileThreads, r = c >> 4;
                        const bool ok = row0 + r < sh.m;
                        cp_async16(base + r * kRowBytes + (c & 15u) * 16u,
                                   x + static_cast<size_t>(ok ? row0 + r : 0u) * sh.k + col + (c & 15u) * 8u, ok);
                    }
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) {
                        const uint32_t c = tid + j * kTileThreads, r = c >> 4;
                        const bool ok = slab + r < sh.rank;
                        if (16u * j >= sh.rank - slab) break;  // 16 rows at a time
                        cp_async16(base + kXBytes + r * kRowBytes + (c & 15u) * 16u,
                                   a_w + (static_cast<size_t>(a) * sh.rank + (ok ? slab + r : 0u)) * sh.k + col + (c & 15u) * 8u, ok);
                    }
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            for (uint32_t i = 0; i < kTileStages - 1; ++i) issue(i);
            // Warp w: rows 16(w%4) .. +15, columns 32(w/4) .. +31 of the slab.
            float acc[4][4] = {};
            const uint32_t mrow = (warp & 3u) * 16u, ncol = (warp >> 2) * 32u;
            const uint32_t columns = sh.rank - slab;  // of A, from this slab on
            for (uint32_t i = 0; g0 + i < g1; ++i) {
                asm volatile("cp.async.wait_group %0;" ::"n"(kTileStages - 2) : "memory");
                __syncthreads();
                issue(i + kTileStages - 1);
                const uint32_t base = smem_addr(sm.stage[i % kTileStages]);
#pragma unroll
                for (uint32_t kk = 0; kk < 8; ++kk) {
                    uint32_t fx[4];
                    ldmatrix_x4(fx, base + (mrow + (lane & 15u)) * kRowBytes + kk * 32u + (lane >> 4) * 16u);
#pragma unroll
                    for (uint32_t n = 0; n < 2; ++n) {
                        if (ncol + 16u * n >= columns) break;
                        uint32_t fa[4];
                        ldmatrix_x4(fa, base + kXBytes + (ncol + 16u * n + (lane & 7u) + ((lane >> 4) << 3)) * kRowBytes + kk * 32u + ((lane >> 3) & 1u) * 16u);
                        mma_bf16_16816(acc[2 * n], fx, fa[0], fa[1]);
                        mma_bf16_16816(acc[2 * n + 1], fx, fa[2], fa[3]);
                    }
                }
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            float(*part)[kSlab] = reinterpret_cast<float(*)[kSlab]>(sm.stage[0]);
            __syncthreads();  // every warp is done with the stages, which hold the sums now
#pragma unroll
            for (uint32_t n = 0; n < 4; ++n)
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h)
                    *reinterpret_cast<float2*>(&part[mrow + h * 8u + (lane >> 2)][ncol + n * 8u + (lane & 3u) * 2u]) =
                        make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
            cluster_sync_all();
            const float scale = __ldg(scaling + a);
            for (uint32_t i = rank * kTileThreads + tid; i < kTileRows * kSlab / 2; i += split * kTileThreads) {
                const uint32_t r = i / (kSlab / 2), c = i % (kSlab / 2) * 2u;
                // The parts are multiplied 16 at a time; past the rank the sums are zero.
                if (sm.ids[r] != a || slab + c >= (sh.v_fp32 ? sh.rank : v_parts(sh.rank) / 2u)) continue;
                float2 n[kTileMaxSplit];
#pragma unroll
                for (uint32_t p = 0; p < kTileMaxSplit; ++p) {
                    n[p] = make_float2(0.0f, 0.0f);
                    if (p < split)
                        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(n[p].x), "=f"(n[p].y) : "r"(mapa_shared(smem_addr(&part[r][c]), p)) : "memory");
                }
                float sx = 0.0f, sy = 0.0f;
#pragma unroll
                for (uint32_t p = 0; p < kTileMaxSplit; ++p) {
                    sx += n[p].x;
                    sy += n[p].y;
                }
                sx *= scale;
                sy *= scale;
                const size_t row = row0 + r;
                if (sh.v_fp32) {
                    *reinterpret_cast<float2*>(static_cast<float*>(v) + row * sh.rank + slab + c) = make_float2(sx, sy);
                } else {
                    uint16_t* to = static_cast<uint16_t*>(v) + row * v_parts(sh.rank) + (slab + c) / 16u * 32u + c % 16u;
                    const uint32_t hi = pack_bf16x2(sx, sy);
                    const float hx = __uint_as_float(hi << 16), hy = __uint_as_float(hi & 0xFFFF0000u);
                    // what an infinity leaves is nothing, not NaN
                    *reinterpret_cast<uint32_t*>(to) = hi;
                    *reinterpret_cast<uint32_t*>(to + 16) = pack_bf16x2(isfinite(hx) ? sx - hx : 0.0f, isfinite(hy) ? sy - hy : 0.0f);
                }
            }
            cluster_sync_all();  // the parts may be overwritten, or the CTA leave
        }
    }
}

}  // namespace

cudaError_t launch_lora_prep(const LoraPrepLaunch& L, uint32_t sms, cudaStream_t stream) {
    PrepShape sh{L.m, L.n, L.k, L.mp, L.adapters, L.rank, 1, L.v_fp32 ? 1u : 0u};
    const uint32_t G = L.k / 128u;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e;
    // A row's part of x lies in shared memory: up to k = 192512 (rank 256) without an opt-in.
    const uint32_t row_split = G < kRowMaxSplit ? G : kRowMaxSplit;
    const size_t row_bytes = static_cast<size_t>(G + row_split - 1) / row_split * 256u + L.rank * sizeof(float);
    if (L.m <= kDecodeMaxTokens && row_bytes <= 48u * 1024u) {
        const uint32_t split = row_split;
        attr[0].val.clusterDim.x = split;
        cfg.gridDim = dim3(L.m * split, 1, 1);
        cfg.blockDim = dim3(kRowThreads, 1, 1);
        cfg.dynamicSmemBytes = row_bytes;
        e = cudaLaunchKernelEx(&cfg, lora_rows_kernel, static_cast<const uint16_t*>(L.x), L.ids,
                               static_cast<const uint16_t*>(L.a), static_cast<const uint16_t*>(L.b), L.scaling,
                               static_cast<uint8_t*>(L.q), L.s_k, static_cast<float*>(L.v), split, sh);
    } else {
        static std::once_flag once[64];
        static cudaError_t optin[64];
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        std::call_once(once[dev], [dev] {
            optin[dev] = cudaFuncSetAttribute(lora_tiles_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                              static_cast<int>(sizeof(TileSmem)));
        });
        if (optin[dev] != cudaSuccess) return optin[dev];
        const uint32_t blocks = (L.m + kTileRows - 1) / kTileRows;
        // One to two CTAs per SM for v, the rest of the SM for the quantizing ones.
        uint32_t split = 1;
        while (split < kTileMaxSplit && split * 2 <= G && blocks * split <= sms) split *= 2;
        const uint32_t parts = (team_parts(L.m * G) + split - 1) / split;
        // As many clusters per 64 rows as there can be passes, but no more CTAs in all
        // than kPassCtas per SM (most have nothing to do when adapters are few).
        const uint32_t most = (L.adapters < kTileRows ? L.adapters : kTileRows) * ((L.rank + kSlab - 1) / kSlab);
        sh.passes = kPassCtas * sms / (blocks * split);
        if (sh.passes < 2) sh.passes = 2;
        if (sh.passes > most) sh.passes = most;
        attr[0].val.clusterDim.x = split;
        cfg.gridDim = dim3((sh.passes * blocks + parts) * split, 1, 1);
        cfg.blockDim = dim3(kTileThreads, 1, 1);
        cfg.dynamicSmemBytes = sizeof(TileSmem);
        e = cudaLaunchKernelEx(&cfg, lora_tiles_kernel, static_cast<const uint16_t*>(L.x), L.ids,
                               static_cast<const uint16_t*>(L.a), L.scaling, static_cast<uint8_t*>(L.q), L.s_k,
                               L.v, L.lists, split, sh);
    }
    note_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace fp8q
