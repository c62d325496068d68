// Block-scaled FP8 projection grouped by expert, ragged groups.
//
//   y[i][c] = bf16( sum_g a_s[r][g] * w_s[e][c/128][g] * P_g[i][c] ),
//   P_g[i][c] = sum_{j<128} q[r][128g+j] * wq[e][c][128g+j]
//
// for the grouped rows i of expert e (offsets[e] <= i < offsets[e+1]), r =
// rows[i] (or i). The arithmetic of a row is the plain projection's: FP8
// tensor-core products per 128-wide K block in fp32, promoted into fp32
// register accumulators with the product of the two scales.
//
// The quantizer writes the codes in grouped order, a row once per slot that uses
// it, so that a block of rows is a plain tile: fetching the rows of ungrouped codes
// by row-gathering TMA loads took 617 us against 400 at 1168 tokens x 8 choices, 64
// experts, N = 4096, K = 5120 (twenty such loads per K block and CTA).
//
// Two kernels on CTA pairs (clusters of 2, one CTA per SM, cta_group::2 MMAs):
//   grouped_tokens_kernel  few rows per expert: weights are the MMA's M (256 rows of
//                          one expert per pair), a block of rows its N, 32 to
//                          kTokens wide, so a group of 70 rows costs 96 columns and
//                          not 256. An expert's rows are cut into equal blocks.
//   grouped_rows_kernel    many: 256 rows on M, 256 weight columns on N.
// Per CTA, 12 warps:
//   warp 0      TMA producer, one barrier for all that a K block needs
//   warps 1, 2  in the even CTA, MMA issuers: of the even and odd K blocks (tokens
//               kernel), of the two column halves (rows kernel)
//   warp 3      idle after set-up
//   warps 4-11  promotion and epilogue: warp w owns TMEM lanes 32*(w%4)..+31 and half
//               of the columns. TMEM loads are in flight while earlier ones are
//               promoted, and a TMEM buffer is handed back as soon as it is read:
//               with operands at hand, what bounds a K block is a buffer's way
//               through the MMA (its work and some 430 clocks), the loads (400) and
//               the barriers between, not the tensor cores (40 % busy at 146 rows
//               per expert).
// The tokens kernel's TMEM loads are fragment-shaped (16 lanes x 16 columns): a
// thread gets two neighbouring tokens of four weight rows, so that a token's scale
// is read once for four rows and the transposing matrix store turns the bf16 tile
// token-major.
//
// Work. The tiles (expert, 256 weight rows, row block) are numbered expert by expert
// with the row block fastest, so that pairs running together share an expert's
// weights and rows in L2. Pair p takes tiles p, p + P, ... Where that would leave many
// pairs idle for long at the end (kSplitCost; few tiles of a long K), the K blocks of
// all tiles form one line that is cut into P equal pieces instead; a pair whose piece ends inside a tile writes its fp32 partial
// to the workspace, and the last of the tile's pairs to arrive (an atomic counter per
// warp) adds the partials in K order, so the sum does not depend on which that is. No
// CTA waits for another pair.
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "group_quant.cuh"
#include "grouped.cuh"
#include "internal.h"
#include "ptx.cuh"
#include "ptx_routed.cuh"
#include "routed.h"
#include "team_quant.cuh"

namespace fp8q {

// Device error word of the grouped projection: bit 3 of fp8q_device_error,
// a CTA gave up on a bounded wait.
__device__ uint32_t g_grouped_error = 0;
constexpr uint32_t kGroupedErrorBit = 8u;

namespace {

constexpr uint32_t BW = 128;       // weight rows per CTA
constexpr uint32_t BW_PAIR = 256;  // weight rows per CTA pair (one MMA)
constexpr uint32_t BK = 128;
constexpr uint32_t kThreads = kGroupedThreads;
constexpr uint32_t kEpiWarps = 8;
constexpr long long kDrainBudget = 20000000;  // clocks that a copy in flight is waited for after a timeout
constexpr uint32_t kChunk = 16;  // tokens of one TMEM load
// 128*56 + 256*224 = 64512 = 384 * 168, the launch allocation.
constexpr uint32_t kRegsLow = 56;
constexpr uint32_t kRegsHigh = 224;
constexpr uint32_t kLaunchRegsNeeded = (128 * kRegsLow + 256 * kRegsHigh + kThreads - 1) / kThreads;

// ------------------------------------------------- few rows per expert --

template <uint32_t kTokens>  // rows of a block, at most
struct TokensConfig {
    static constexpr uint32_t kTokenBytes = kTokens / 2 * BK;  // one CTA's half of them
    static constexpr uint32_t kStages = kTokens > 64 ? 8 : 10;
    static constexpr uint32_t kBufs = 512 / kTokens;
    static constexpr uint32_t kChunks = kTokens / kChunk / 2;  // per promotion warp
    // A K block's token scales start at a multiple of four rows (16 bytes).
    static constexpr uint32_t kScaleBox = kTokens + 4;
    // A scale slot is free again once the promotion of its K block has handed its
    // TMEM buffer back. The producer fills the stage of K block i after MMA
    // i - kStages, which waited for the buffer of K block i - kStages - kBufs: with
    // that many slots no barrier of their own is needed.
    static constexpr uint32_t kScaleSlots = kStages + kBufs;
    static_assert(kStages % 2 == 0, "each stage must always be consumed by the same MMA issuer");
};

template <uint32_t kTokens>
struct __align__(1024) TokensSmem {
    using C = TokensConfig<kTokens>;
    uint8_t w[C::kStages][BW * BK];
    uint8_t t[C::kStages][C::kTokenBytes];
    uint8_t out[kEpiWarps][8 * 64];
    alignas(128) float scale[C::kScaleSlots][(C::kScaleBox + 31) / 32 * 32];
    uint64_t full[C::kStages];
    uint64_t empty[C::kStages];
    uint64_t tfull[C::kBufs];
    uint64_t tempty[C::kBufs];
    uint64_t mma_done[2];
    uint32_t tmem_base;
    uint32_t abort;
    uint32_t consumed[2];
    Experts experts;
};

template <uint32_t kTokens>
constexpr size_t tokens_smem_bytes() {
    static_assert(sizeof(TokensSmem<kTokens>) + 1024 <= 232448, "shared memory of a CTA");
    return sizeof(TokensSmem<kTokens>) + 1024;
}

// MMA N of a block: its rows rounded up to 32.
__device__ __forceinline__ uint32_t width_of(const Piece& w) { return (w.rows + 31u) & ~31u; }

// Scales of a thread's tokens of kChunks chunks, times the weight block's.
template <uint32_t kChunks>
__device__ __forceinline__ void read_scales(const float* from, float w, float2 (&a)[kChunks][2]) {
#pragma unroll
    for (uint32_t c = 0; c < kChunks; ++c)
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j)
            a[c][j] = __fmul2_rn(make_float2(from[16u * c + 8u * j], from[16u * c + 8u * j + 1u]), make_float2(w, w));
}

// acc += a * v for the kChunks chunks of v.
template <uint32_t kChunks, uint32_t kAll>
__device__ __forceinline__ void add_scaled(const float2 (&a)[kChunks][2], const uint32_t (&v)[16 * kChunks], uint32_t first,
                                           float2 (&acc)[kAll][2][2][2]) {
#pragma unroll
    for (uint32_t c = 0; c < kChunks; ++c)
#pragma unroll
        for (uint32_t j = 0; j < 2; ++j)
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h)
#pragma unroll
                for (uint32_t r = 0; r < 2; ++r) {
                    const uint32_t at = tmem_frag<kChunks>(c, h, j) + 2 * r;
                    acc[first + c][h][j][r] = __ffma2_rn(a[c][j], make_float2(__uint_as_float(v[at]), __uint_as_float(v[at + 1])),
                                                         acc[first + c][h][j][r]);
                }
}

// The promotion of one warp's part of a tile: `count` K blocks, kMine chunks of
// tokens (one past the block is promoted too, and never stored: a test of the
// block's width around each chunk made the loop twice as slow). The chunks are
// taken in two parts, each part's TMEM load in flight while the other is promoted,
// across K blocks too. `tmem` names this warp's lanes and first column, `token`
// this lane's first token in a scale slot, `ws` the weight block's scales (null:
// per-row weights). False when a wait gave up.
template <uint32_t kMine, uint32_t kTokens>
__device__ __forceinline__ bool promote(TokensSmem<kTokens>& sm, Ring<TokensConfig<kTokens>::kBufs>& buf,
                                        Ring<TokensConfig<kTokens>::kScaleSlots>& slot, uint32_t count, uint32_t tmem, uint32_t token,
                                        const float* ws, uint32_t lane, uint32_t tempty_even, long long budget,
                                        float2 (&acc)[TokensConfig<kTokens>::kChunks][2][2][2]) {
    constexpr uint32_t kFirst = (kMine + 1) / 2, kSecond = kMine - kFirst;
    uint32_t v0[16 * kFirst], v1[16 * kSecond];
    float2 a0[kFirst][2], a1[kSecond][2];
    float w = ws ? __ldg(ws) : 1.0f;
    // The K block's products and scales have landed; the first part on its way.
    auto begin = [&]() {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sm.tfull[buf.slot], buf.phase, &sm.abort, budget))) return false;
        tc_fence_after();
        tmem_load_frags<kFirst>(tmem + buf.slot * kTokens, v0);
        read_scales<kFirst>(sm.scale[slot.slot] + token, w, a0);
        return true;
    };
    if (!begin()) return false;
    for (;;) {
        const uint32_t b = buf.slot;
        tmem_wait_frags(v0);
        tmem_load_frags<kSecond>(tmem + b * kTokens + kFirst * kChunk, v1);
        read_scales<kSecond>(sm.scale[slot.slot] + token + kFirst * kChunk, w, a1);
        if (ws && count > 1) w = __ldg(++ws);
        add_scaled<kFirst>(a0, v0, 0, acc);
        tmem_wait_frags(v1);
        // The buffer and the scales have been read.
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty_even + b * 8u);
        buf.step();
        slot.step();
        if (--count != 0 && !begin()) return false;
        add_scaled<kSecond>(a1, v1, kFirst, acc);
        if (count == 0) return true;
    }
}

template <uint32_t kTokens>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    grouped_tokens_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT,
                        const __grid_constant__ CUtensorMap tmS, const float* __restrict__ w_s,
                        const int32_t* __restrict__ offsets, uint16_t* __restrict__ y,
                        float* __restrict__ partial, uint32_t* __restrict__ counters, const GroupedShape sh) {
    using C = TokensConfig<kTokens>;
    using TokensWalk = Walk<kTokens, true>;
    extern __shared__ uint8_t smem_raw[];
    TokensSmem<kTokens>& sm = *reinterpret_cast<TokensSmem<kTokens>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t pair = blockIdx.x >> 1;
    const uint32_t num_pairs = gridDim.x >> 1;
    volatile uint32_t* abort = &sm.abort;

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < C::kStages; ++s) {
            mbar_init(&sm.full[s], 2);  // one expect-tx arrival from each CTA of the pair
            mbar_init(&sm.empty[s], 1);
        }
        for (uint32_t b = 0; b < C::kBufs; ++b) {
            mbar_init(&sm.tfull[b], 1);
            mbar_init(&sm.tempty[b], 2 * kEpiWarps);  // promotion warps of both CTAs
        }
        mbar_init(&sm.mma_done[0], 1);
        mbar_init(&sm.mma_done[1], 1);
        sm.abort = 0;
        sm.consumed[0] = sm.consumed[1] = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmT);
        tma_prefetch_desc(&tmS);
    }
    if (warp == 1) {
        tmem_alloc_pair(&sm.tmem_base, 512);
        tmem_relinquish_pair();
    }
    // The grid before this one is the quantizer of the rows, which let this one
    // start after everything before it had completed: the offsets and the weights
    // may be read at once, so the first stages' weights are on their way while the
    // rows are quantized. Codes, scales and counters are the quantizer's.
    list_experts<kTokens>(sm.experts, offsets, sh);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // barriers of both CTAs initialised before any remote arrive
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;

    uint32_t issued = 0;  // producer: K blocks whose loads were all issued

    if (warp < 4) {
        regs_dec<kRegsLow>();
        TokensWalk walk(sm.experts, sh, pair, num_pairs);
        Piece w;
        if (warp == 0 && !sh.no_copies) {
            auto weight_row = [&](const Piece& p) {
                return static_cast<int32_t>(p.expert * sh.N + (p.n0 + rank * BW < sh.N ? p.n0 + rank * BW : p.n0));
            };
            // A stage's bytes are announced with its weights; rows past the block are
            // the next expert's or, past the last row, zero.
            auto load_weights = [&](uint32_t s, const Piece& p, uint32_t kb) {
                const uint32_t full_even = mapa_shared(smem_addr(&sm.full[s]), 0);
                mbar_arrive_expect_tx_cluster(full_even, BW * BK + width_of(p) / 2u * BK + C::kScaleBox * 4u);
                tma_load_2d_pair(sm.w[s], &tmW, full_even, static_cast<int32_t>(kb * BK), weight_row(p));
            };
            uint32_t early = 0;
            {
                TokensWalk ahead(sm.experts, sh, pair, num_pairs);
                while (early < C::kStages && ahead.pop(w))
                    for (uint32_t kb = w.kb0; kb < w.kb1 && early < C::kStages; ++kb, ++early)
                        if (elect_one()) load_weights(early, w, kb);
                __syncwarp();
            }
            grid_dependency_wait();
            uint32_t it = 0;
            bool ok = true;
            while (ok && walk.pop(w)) {
                // This CTA stages tokens half .. half + width/2 - 1 of the block.
                const uint32_t half = width_of(w) / 2u;
                const int32_t first = static_cast<int32_t>(w.row0 + rank * half);
                for (uint32_t kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    const uint32_t s = it % C::kStages;
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sm.empty[s], ((it / C::kStages) & 1u) ^ 1u, abort, sh.budget))) {
                        ok = false;
                        break;
                    }
                    if (elect_one()) {
                        if (it >= early) load_weights(s, w, kb);
                        const uint32_t full_even = mapa_shared(smem_addr(&sm.full[s]), 0);
                        const int32_t kx = static_cast<int32_t>(kb * BK);
                        for (uint32_t r = 0; r < half; r += 16u)
                            tma_load_2d_pair(sm.t[s] + r * BK, &tmT, full_even, kx, first + static_cast<int32_t>(r));
                        tma_load_2d_pair(sm.scale[it % C::kScaleSlots], &tmS, full_even, static_cast<int32_t>(w.row0 & ~3u), static_cast<int32_t>(kb));
                    }
                    __syncwarp();
                    issued = it + 1;
                }
            }
        } else if ((warp == 1 || warp == 2) && rank == 0) {
            // Two MMA issuers, by K-block parity, as in the plain projection.
            const uint32_t par = warp - 1u;
            uint32_t it = 0;
            bool ok = true;
            while (ok && walk.pop(w)) {
                const uint32_t idesc = idesc_e4m3_f32(BW_PAIR, width_of(w));
                for (uint32_t kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    if ((it & 1u) != par) continue;
                    const uint32_t s = it % C::kStages;
                    const uint32_t ph = (it / C::kStages) & 1u;
                    const uint32_t b = it % C::kBufs;
                    const uint32_t tph = (it / C::kBufs) & 1u;
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sm.full[s], ph, abort, sh.budget))) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) sm.consumed[par] = it + 1;
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sm.tempty[b], tph ^ 1u, abort, sh.budget))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + b * kTokens;
                    const uint64_t ad = smem_desc_k_sw128(smem_addr(sm.w[s]));
                    const uint64_t bd = smem_desc_k_sw128(smem_addr(sm.t[s]));
                    if (elect_one()) {
#pragma unroll
                        for (uint32_t kk = 0; kk < BK / 32; ++kk)
                            mma_f8f6f4_pair(d, ad + 2u * kk, bd + 2u * kk, idesc, kk > 0 ? 1u : 0u);
                        mma_commit_pair_multicast(&sm.tfull[b], 0x3);
                        mma_commit_pair_multicast(&sm.empty[s], 0x3);
                    }
                    __syncwarp();
                }
            }
            // Every MMA this thread issued has completed once mma_done fires.
            if (elect_one()) mma_commit_pair(&sm.mma_done[par]);
            __syncwarp();
            volatile uint32_t never = 0;
            mbar_wait(&sm.mma_done[par], 0, &never);
        }
    } else {
        regs_inc<kRegsHigh>();
        grid_dependency_wait();  // the counters are the quantizer's
        TokensWalk walk(sm.experts, sh, pair, num_pairs);
        Piece w;
        const uint32_t quad = warp & 3u;
        const uint32_t side = (warp - 4u) >> 2;  // which half of the tokens
        const uint32_t lane_off = (quad * 32u) << 16;
        uint8_t* stg = sm.out[warp - 4u];
        const uint32_t tempty_even = mapa_shared(smem_addr(&sm.tempty[0]), 0);
        Ring<C::kBufs> buf;
        Ring<C::kScaleSlots> slot;
        while (walk.pop(w)) {
            // acc[c][h][j][r]: tokens half0 + 16c + 8j + 2*(lane%4), +1 of weight row 16h + 8r + lane/4
            float2 acc[C::kChunks][2][2][2];
#pragma unroll
            for (uint32_t c = 0; c < C::kChunks; ++c)
#pragma unroll
                for (uint32_t i = 0; i < 8; ++i) acc[c][i >> 2][(i >> 1) & 1][i & 1] = make_float2(0.0f, 0.0f);
            const uint32_t half0 = side * (width_of(w) / 2u);
            const uint32_t chunks = width_of(w) / (2u * kChunk);
            const uint32_t count = w.kb1 - w.kb0;
            const uint32_t wn = w.n0 + rank * BW < sh.N ? w.n0 + rank * BW : w.n0;
            const float* ws = sh.w_per_row ? nullptr : w_s + (static_cast<size_t>(w.expert) * (sh.N / BW) + wn / BW) * sh.G + w.kb0;
            const uint32_t token = (w.row0 & 3u) + half0 + 2u * (lane & 3u);
            const uint32_t lanes = tmem + lane_off + half0;
            bool ok;
            if constexpr (C::kChunks <= 3) ok = promote<C::kChunks>(sm, buf, slot, count, lanes, token, ws, lane, tempty_even, sh.budget, acc);
            else if (chunks <= 3) ok = promote<3>(sm, buf, slot, count, lanes, token, ws, lane, tempty_even, sh.budget, acc);
            else ok = promote<C::kChunks>(sm, buf, slot, count, lanes, token, ws, lane, tempty_even, sh.budget, acc);
            if (!ok) break;
            const uint32_t n_first = w.n0 + rank * BW + quad * 32u;
            if (n_first >= sh.N) continue;
            if (w.kb1 - w.kb0 < sh.G) {
                // A part of the tile's K range: park it, and let the warp that
                // comes last add up all parts in K order.
                const Partial<C::kChunks * 4> part{reinterpret_cast<float4*>(partial), &counters[(w.tile * 2u + rank) * kEpiWarps + (warp - 4u)], pair,
                                                walk.owner(w.tile * sh.G), walk.owner(w.tile * sh.G + sh.G - 1u), rank, warp - 4u, lane};
#pragma unroll
                for (uint32_t c = 0; c < C::kChunks; ++c)
                    if (c < chunks)
#pragma unroll
                        for (uint32_t i = 0; i < 4; ++i) {
                            const float2 a0 = acc[c][i >> 1][i & 1][0], a1 = acc[c][i >> 1][i & 1][1];
                            part.put(c * 4u + i, make_float4(a0.x, a0.y, a1.x, a1.y));
                        }
                if (!part.last()) continue;
#pragma unroll
                for (uint32_t c = 0; c < C::kChunks; ++c)
                    if (c < chunks) {
                        float4 sum[4];
                        part.sum(c * 4u, sum);
#pragma unroll
                        for (uint32_t i = 0; i < 4; ++i) {
                            acc[c][i >> 1][i & 1][0] = make_float2(sum[i].x, sum[i].y);
                            acc[c][i >> 1][i & 1][1] = make_float2(sum[i].z, sum[i].w);
                        }
                    }
            }
            float row_scale[2][2];
#pragma unroll
            for (uint32_t h = 0; h < 2; ++h)
#pragma unroll
                for (uint32_t r = 0; r < 2; ++r)
                    row_scale[h][r] = sh.w_per_row ? __ldg(w_s + static_cast<size_t>(w.expert) * sh.N + n_first + 16u * h + 8u * r + (lane >> 2)) : 1.0f;
            // 8 tokens x 32 weight rows at a time: packed to bf16, turned to
            // token-major rows of 64 bytes (16-byte piece j of row t at piece
            // j ^ ((t >> 1) & 3), free of bank conflicts both ways), and written
            // 16 bytes a lane. Rows past the block belong to the next expert
            // and are not written.
            const uint32_t t = lane & 7u, u = lane >> 2;
            const uint32_t to = smem_addr(stg) + t * 64u + (((lane >> 3) ^ ((t >> 1) & 3u)) << 4);
            const uint4* from = reinterpret_cast<const uint4*>(stg + u * 64u + (((lane & 3u) ^ ((u >> 1) & 3u)) << 4));
            uint16_t* out = y + static_cast<size_t>(w.row0 + half0 + u) * sh.N + n_first + (lane & 3u) * 8u;
#pragma unroll
            for (uint32_t c = 0; c < C::kChunks; ++c) {
                if (c >= chunks) break;
#pragma unroll
                for (uint32_t j = 0; j < 2; ++j) {
                    uint32_t p[4];
#pragma unroll
                    for (uint32_t i = 0; i < 4; ++i) {
                        const float2 a = acc[c][i >> 1][j][i & 1];
                        const float s = row_scale[i >> 1][i & 1];
                        p[i] = pack_bf16x2(a.x * s, a.y * s);
                    }
                    __syncwarp();
                    stmatrix_x4_trans(to, p[0], p[1], p[2], p[3]);
                    __syncwarp();
                    const uint32_t at = c * kChunk + 8u * j;
                    if (half0 + at + u < w.rows) *reinterpret_cast<uint4*>(out + static_cast<size_t>(at) * sh.N) = *from;
                }
            }
        }
    }

    // Teardown, as in the plain projection: after a timed-out wait the loads
    // this pair started may still be landing, so they are waited for (bounded)
    // before the pair synchronises and frees TMEM.
    tc_fence_before();
    __syncthreads();
    if (*abort) {
        volatile uint32_t never = 0;
        if (threadIdx.x == 0) atomicOr(&g_grouped_error, kGroupedErrorBit);
        if (warp == 0 && lane == 0) {
            if (rank == 0) {
                const uint32_t from = sm.consumed[0] < sm.consumed[1] ? sm.consumed[0] : sm.consumed[1];
                for (uint32_t it = from; it < issued; ++it)
                    if (it >= sm.consumed[it & 1u]) mbar_wait(&sm.full[it % C::kStages], (it / C::kStages) & 1u, &never, kDrainBudget);
            }
            const long long t0 = clock64();
            while (clock64() - t0 < 200000) {
            }
        }
        __syncthreads();
    }
    cluster_sync_all();  // no remote arrive or pair MMA can still target this CTA
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

// ------------------------------------------------ many rows per expert --
//
// The plain projection's orientation: rows on the MMA's M (256 per pair), 256
// weight columns on its N, one row's accumulators per thread and column half.
// A row's scale is then one number per thread. A K block is multiplied in two
// halves of 128 columns, each with its own issuing warp, TMEM buffers and four
// promotion warps. What bounds the loop is a buffer's way through the MMA (about
// 430 clocks more than its work) and the promotion (700 clocks until the buffer is
// read); halves out of step overlap a little of it (a 5120-column layer of 64
// experts at 146 rows each, 218 us in one piece and 214 in halves).

constexpr uint32_t BM = 128;  // rows per CTA
constexpr uint32_t BM_PAIR = 256;
constexpr uint32_t BN = 256;
constexpr uint32_t BN_CTA = 128;
constexpr uint32_t kRowStages = 5;
constexpr uint32_t kOutCols = 64;  // columns of one output store

struct __align__(1024) RowsSmem {
    uint8_t a[kRowStages][BM * BK];
    uint8_t b[kRowStages][BN_CTA * BK];
    uint8_t out[kEpiWarps][32 * kOutCols * 2];
    uint64_t full[kRowStages];
    uint64_t empty[kRowStages];
    uint64_t tfull[2][2];   // [half][buffer]
    uint64_t tempty[2][2];
    uint64_t mma_done[2];
    uint32_t tmem_base;
    uint32_t abort;
    uint32_t consumed[2];
    Experts experts;
};
static_assert(sizeof(RowsSmem) + 1024 <= 232448, "shared memory of a CTA");

using RowsWalk = Walk<BM_PAIR, false>;

// acc += c * v, 32 columns.
__device__ __forceinline__ void add_part(float c, const uint32_t (&v)[32], float2 (&acc)[16]) {
    const float2 c2 = make_float2(c, c);
#pragma unroll
    for (uint32_t i = 0; i < 16; ++i)
        acc[i] = __ffma2_rn(c2, make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), acc[i]);
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    grouped_rows_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                        const __grid_constant__ CUtensorMap tmY, const float* __restrict__ s_k,
                        const float* __restrict__ w_s, const int32_t* __restrict__ offsets, uint16_t* __restrict__ y,
                        float* __restrict__ partial, uint32_t* __restrict__ counters, const GroupedShape sh) {
    extern __shared__ uint8_t smem_raw[];
    RowsSmem& sm = *reinterpret_cast<RowsSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0);
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const uint32_t pair = blockIdx.x >> 1;
    const uint32_t num_pairs = gridDim.x >> 1;
    volatile uint32_t* abort = &sm.abort;

    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < kRowStages; ++s) {
            mbar_init(&sm.full[s], 2);  // one expect-tx arrival from each CTA of the pair
            mbar_init(&sm.empty[s], 2);  // the MMAs of both halves
        }
        for (uint32_t h = 0; h < 2; ++h) {
            for (uint32_t b = 0; b < 2; ++b) {
                mbar_init(&sm.tfull[h][b], 1);
                mbar_init(&sm.tempty[h][b], kEpiWarps);  // the half's four promotion warps of both CTAs
            }
            mbar_init(&sm.mma_done[h], 1);
        }
        sm.abort = 0;
        sm.consumed[0] = sm.consumed[1] = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
        tma_prefetch_desc(&tmY);
    }
    if (warp == 1) {
        tmem_alloc_pair(&sm.tmem_base, 2 * BN);
        tmem_relinquish_pair();
    }
    // The offsets may come from the grid before this one.
    grid_dependency_wait();
    list_experts<BM_PAIR>(sm.experts, offsets, sh);
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();  // barriers of both CTAs initialised before any remote arrive
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;

    uint32_t issued = 0;  // producer: K blocks whose loads were issued

    if (warp < 4) {
        regs_dec<kRegsLow>();
        RowsWalk walk(sm.experts, sh, pair, num_pairs);
        Piece w;
        if (warp == 0 && !sh.no_copies) {
            uint32_t it = 0;
            bool ok = true;
            while (ok && walk.pop(w)) {
                const int32_t my_m = static_cast<int32_t>(w.row0 + rank * BM);
                // Half h of the columns is rows 64h .. 64h + 63 of both CTAs' weight tiles.
                const int32_t my_n = static_cast<int32_t>(w.expert * sh.N + w.n0 + rank * 64u);
                // A CTA whose 128 rows all lie past the block loads none; its accumulators are not read.
                const bool rows = w.rows > rank * BM;
                for (uint32_t kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    const uint32_t s = it % kRowStages;
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sm.empty[s], ((it / kRowStages) & 1u) ^ 1u, abort, sh.budget))) {
                        ok = false;
                        break;
                    }
                    const uint32_t full_even = mapa_shared(smem_addr(&sm.full[s]), 0);
                    const int32_t kx = static_cast<int32_t>(kb * BK);
                    if (elect_one()) {
                        mbar_arrive_expect_tx_cluster(full_even, (rows ? BM * BK : 0u) + BN_CTA * BK);
                        if (rows) tma_load_2d_pair(sm.a[s], &tmA, full_even, kx, my_m);
                        tma_load_2d_pair(sm.b[s], &tmB, full_even, kx, my_n);
                        tma_load_2d_pair(sm.b[s] + 64u * BK, &tmB, full_even, kx, my_n + 128);
                    }
                    __syncwarp();
                    issued = it + 1;
                }
            }
        } else if ((warp == 1 || warp == 2) && rank == 0) {
            // One MMA issuer per half.
            constexpr uint32_t idesc = idesc_e4m3_f32(BM_PAIR, BN / 2);
            const uint32_t h = warp - 1u;
            uint32_t it = 0;
            bool ok = true;
            while (ok && walk.pop(w)) {
                for (uint32_t kb = w.kb0; kb < w.kb1; ++kb, ++it) {
                    const uint32_t s = it % kRowStages;
                    const uint32_t b = it & 1u;
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sm.full[s], (it / kRowStages) & 1u, abort, sh.budget))) {
                        ok = false;
                        break;
                    }
                    if (lane == 0) sm.consumed[h] = it + 1;
                    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sm.tempty[h][b], ((it >> 1) & 1u) ^ 1u, abort, sh.budget))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t d = tmem + b * BN + h * 128u;
                    const uint64_t ad = smem_desc_k_sw128(smem_addr(sm.a[s]));
                    const uint64_t bd = smem_desc_k_sw128(smem_addr(sm.b[s] + h * 64u * BK));
                    if (elect_one()) {
#pragma unroll
                        for (uint32_t kk = 0; kk < BK / 32; ++kk)
                            mma_f8f6f4_pair(d, ad + 2u * kk, bd + 2u * kk, idesc, kk > 0 ? 1u : 0u);
                        mma_commit_pair_multicast(&sm.tfull[h][b], 0x3);
                        mma_commit_pair_multicast(&sm.empty[s], 0x3);
                    }
                    __syncwarp();
                }
            }
            // Every MMA this thread issued has completed once mma_done fires.
            if (elect_one()) mma_commit_pair(&sm.mma_done[h]);
            __syncwarp();
            volatile uint32_t never = 0;
            mbar_wait(&sm.mma_done[h], 0, &never);
        }
    } else {
        regs_inc<kRegsHigh>();
        RowsWalk walk(sm.experts, sh, pair, num_pairs);
        Piece w;
        const uint32_t quad = warp & 3u;
        const uint32_t half = (warp - 4u) >> 2;
        const uint32_t lanes = tmem + ((quad * 32u) << 16) + half * 128u;
        const uint32_t tempty_even = mapa_shared(smem_addr(&sm.tempty[half][0]), 0);
        uint8_t* stg = sm.out[warp - 4u];
        Ring<2> buf;
        bool ok = true;
        while (ok && walk.pop(w)) {
            const uint32_t first = rank * BM + quad * 32u;  // this warp's first row in the block
            const uint32_t rows = w.rows > first ? w.rows - first : 0u;
            const uint32_t col0 = w.n0 + half * 128u;
            const bool live = rows != 0 && col0 < sh.N;
            uint32_t count = w.kb1 - w.kb0;
            auto release = [&]() {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(tempty_even + buf.slot * 8u);
                buf.step();
            };
            auto wait = [&]() {
                const bool got = __all_sync(0xFFFFFFFFu, mbar_wait(&sm.tfull[half][buf.slot], buf.phase, abort, sh.budget));
                tc_fence_after();
                return got;
            };
            if (!live) {  // nothing of this tile is the warp's: hand the buffers on
                for (; ok && count != 0; --count) {
                    ok = wait();
                    if (ok) release();
                }
                continue;
            }
            float2 acc[4][16];
#pragma unroll
            for (uint32_t i = 0; i < 64; ++i) acc[i >> 4][i & 15] = make_float2(0.0f, 0.0f);
            // The row's scales are loaded four K blocks ahead; rows past the
            // block have another row's, and are not stored.
            const uint32_t row = min(w.row0 + first + lane, sh.total_pad - 1u);
            const float* a_row = s_k + static_cast<size_t>(w.kb0) * sh.total_pad + row;
            const float* ws = w_s + (sh.w_per_row ? 0u : (static_cast<size_t>(w.expert) * (sh.N / 128u) + col0 / 128u) * sh.G + w.kb0);
            float aq[4];
#pragma unroll
            for (uint32_t i = 0; i < 4; ++i) aq[i] = i < count ? __ldg(a_row + static_cast<size_t>(i) * sh.total_pad) : 0.0f;
            a_row += static_cast<size_t>(4) * sh.total_pad;
            float w_next = sh.w_per_row ? 1.0f : __ldg(ws);
            uint32_t v0[32], v1[32];
            ok = wait();
            if (!ok) break;
            tmem_load32(lanes + buf.slot * BN, v0);
            for (;;) {
                const uint32_t at = lanes + buf.slot * BN;
                const float c = aq[0] * w_next;
                aq[0] = aq[1];
                aq[1] = aq[2];
                aq[2] = aq[3];
                aq[3] = count > 4 ? __ldg(a_row) : 0.0f;
                a_row += sh.total_pad;
                if (!sh.w_per_row && count > 1) w_next = __ldg(++ws);
                // Each 32 columns on their way from TMEM while those before are promoted.
                tmem_wait32(v0);
                tmem_load32(at + 32u, v1);
                add_part(c, v0, acc[0]);
                tmem_wait32(v1);
                tmem_load32(at + 64u, v0);
                add_part(c, v1, acc[1]);
                tmem_wait32(v0);
                tmem_load32(at + 96u, v1);
                add_part(c, v0, acc[2]);
                tmem_wait32(v1);
                release();
                if (--count != 0) {
                    ok = wait();
                    if (!ok) break;
                    tmem_load32(lanes + buf.slot * BN, v0);
                }
                add_part(c, v1, acc[3]);
                if (count == 0) break;
            }
            if (!ok) break;
            if (w.kb1 - w.kb0 < sh.G) {
                // A part of the tile's K range, as above.
                const Partial<32> part{reinterpret_cast<float4*>(partial), &counters[(w.tile * 2u + rank) * kEpiWarps + (warp - 4u)], pair,
                                       walk.owner(w.tile * sh.G), walk.owner(w.tile * sh.G + sh.G - 1u), rank, warp - 4u, lane};
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i) {
                    const float2 a0 = acc[i >> 3][2 * (i & 7)], a1 = acc[i >> 3][2 * (i & 7) + 1];
                    part.put(i, make_float4(a0.x, a0.y, a1.x, a1.y));
                }
                if (!part.last()) continue;
#pragma unroll
                for (uint32_t g = 0; g < 4; ++g) {
                    float4 sum[8];
                    part.sum(g * 8u, sum);
#pragma unroll
                    for (uint32_t i = 0; i < 8; ++i) {
                        acc[g][2 * i] = make_float2(sum[i].x, sum[i].y);
                        acc[g][2 * i + 1] = make_float2(sum[i].z, sum[i].w);
                    }
                }
            }
            if (sh.w_per_row) {
                const float4* wv = reinterpret_cast<const float4*>(w_s + static_cast<size_t>(w.expert) * sh.N + col0);
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i) {
                    const float4 s4 = __ldg(wv + i);
                    float2(&a)[2] = reinterpret_cast<float2(&)[2]>(acc[i >> 3][2 * (i & 7)]);
                    a[0] = __fmul2_rn(a[0], make_float2(s4.x, s4.y));
                    a[1] = __fmul2_rn(a[1], make_float2(s4.z, s4.w));
                }
            }
            // The warp's 32 rows x 128 columns leave as two 32 x 64 blocks (16-byte
            // piece j of row r at piece j ^ (r & 7)) by TMA stores. Of rows that end
            // inside the 32 only the block's own are written, because the ones behind
            // belong to the next expert.
#pragma unroll
            for (uint32_t c = 0; c < 2; ++c) {
                bulk_store_wait_read();  // the block before has left the buffer
                __syncwarp();
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) {
                    const float2* v = &acc[2 * c + (j >> 2)][4 * (j & 3)];
                    *reinterpret_cast<uint4*>(stg + lane * 128u + ((j ^ (lane & 7u)) << 4)) =
                        make_uint4(pack_bf16x2(v[0].x, v[0].y), pack_bf16x2(v[1].x, v[1].y), pack_bf16x2(v[2].x, v[2].y), pack_bf16x2(v[3].x, v[3].y));
                }
                if (rows >= 32) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (elect_one()) tma_store_2d(&tmY, stg, static_cast<int32_t>(col0 + c * kOutCols), static_cast<int32_t>(w.row0 + first));
                } else {
                    __syncwarp();
                    for (uint32_t r = lane >> 3; r < rows; r += 4)
                        *reinterpret_cast<uint4*>(y + static_cast<size_t>(w.row0 + first + r) * sh.N + col0 + c * kOutCols + (lane & 7u) * 8u) =
                            *reinterpret_cast<const uint4*>(stg + r * 128u + (((lane & 7u) ^ (r & 7u)) << 4));
                }
            }
        }
        // Every output block of this warp is in global memory before the CTA
        // (and its staging buffer) goes away.
        bulk_store_wait_all();
        __syncwarp();
    }

    // Teardown, as above.
    tc_fence_before();
    __syncthreads();
    if (*abort) {
        volatile uint32_t never = 0;
        if (threadIdx.x == 0) atomicOr(&g_grouped_error, kGroupedErrorBit);
        if (warp == 0 && lane == 0) {
            if (rank == 0) {
                const uint32_t from = sm.consumed[0] > sm.consumed[1] ? sm.consumed[0] : sm.consumed[1];
                for (uint32_t it = from; it < issued; ++it) mbar_wait(&sm.full[it % kRowStages], (it / kRowStages) & 1u, &never, kDrainBudget);
            }
            const long long t0 = clock64();
            while (clock64() - t0 < 200000) {
            }
        }
        __syncthreads();
    }
    cluster_sync_all();  // no remote arrive or pair MMA can still target this CTA
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 2 * BN);
    }
}

// ---------------------------------------------------------- quantizer --

// Grouped rows to e4m3 codes and K-major scales, eight lanes a group of 128
// (the library's group arithmetic), kQuantGroups groups per eight lanes whose
// loads are in flight together, 128 groups per CTA. Row i is row rows[i] of x
// (row i without `rows`); one that names no row of x gives zero codes and a zero
// scale. The CTAs also clear the counters of the grouped projections that follow.
constexpr uint32_t kQuantGroups = 4;

__global__ void __launch_bounds__(256) quant_rows_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ rows,
                                                         uint8_t* __restrict__ q, float* __restrict__ s_k,
                                                         uint32_t* __restrict__ counters, uint32_t num_counters,
                                                         uint32_t tokens, uint32_t groups, uint32_t G, uint32_t mp) {
    grid_dependency_wait();
    trigger_dependents();
    for (uint32_t i = blockIdx.x * 256u + threadIdx.x; i < num_counters; i += gridDim.x * 256u) counters[i] = 0;
    const uint32_t l = threadIdx.x & 7u;
    uint32_t at[kQuantGroups], row[kQuantGroups];
    uint4 a[kQuantGroups], b[kQuantGroups];
#pragma unroll
    for (uint32_t i = 0; i < kQuantGroups; ++i) {
        at[i] = blockIdx.x * (32u * kQuantGroups) + 32u * i + (threadIdx.x >> 3);
        row[i] = at[i] / G;
        const bool ok = at[i] < groups;
        const uint32_t from = !ok ? tokens : rows ? static_cast<uint32_t>(__ldg(rows + row[i])) : row[i];
        a[i] = b[i] = make_uint4(0u, 0u, 0u, 0u);
        if (from < tokens) {
            const uint16_t* src = x + (static_cast<size_t>(from) * G + (at[i] - row[i] * G)) * 128u + l * 8u;
            a[i] = __ldg(reinterpret_cast<const uint4*>(src));
            b[i] = __ldg(reinterpret_cast<const uint4*>(src + 64));
        } else {
            row[i] |= 0x80000000u;  // no such row
        }
    }
#pragma unroll
    for (uint32_t i = 0; i < kQuantGroups; ++i) {
        uint2 ca, cb;
        const float s = encode_team(a[i], b[i], &ca, &cb);
        if (at[i] < groups) {
            store_team(q + static_cast<size_t>(at[i]) * 128u, l, ca, cb);
            const uint32_t r = row[i] & 0x7FFFFFFFu;
            if (l == 0) s_k[static_cast<size_t>(at[i] - r * G) * mp + r] = row[i] >> 31 ? 0.0f : s;
        }
    }
}

// ----------------------------------------------------------- host side --

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// A [rows, inner] byte matrix read in [box_rows, 128-byte] tiles with the
// 128-byte swizzle.
bool make_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t rows, uint32_t box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {inner, rows};
    cuuint64_t strides[1] = {inner};
    cuuint32_t box[2] = {128, box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The K-major scales [G, padded rows] read `box` tokens of one K group at a time.
bool make_scale_map(CUtensorMap* map, const float* base, uint64_t pad, uint64_t G, uint32_t box_tokens) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {pad, G};
    cuuint64_t strides[1] = {pad * sizeof(float)};
    cuuint32_t box[2] = {box_tokens, 1};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Setup {
    cudaError_t err = cudaSuccess;
    uint32_t pairs = 0;
};

// Once per device: shared-memory opt-in, the register split check, pairs.
const Setup& setup_for_device() {
    static std::mutex mu;
    static Setup table[64];
    static bool done[64] = {};
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= 64) dev = 0;
    std::lock_guard<std::mutex> lock(mu);
    Setup& k = table[dev];
    if (!done[dev]) {
        done[dev] = true;
        auto prepare = [&](const void* fn, size_t bytes) {
            if (k.err == cudaSuccess)
                k.err = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
            cudaFuncAttributes attr;
            if (k.err == cudaSuccess) k.err = cudaFuncGetAttributes(&attr, fn);
            // setmaxnreg.inc waits for registers of the CTA's own allocation.
            if (k.err == cudaSuccess && static_cast<uint32_t>(attr.numRegs) < kLaunchRegsNeeded)
                k.err = cudaErrorInvalidConfiguration;
        };
        prepare(reinterpret_cast<const void*>(grouped_tokens_kernel<64>), tokens_smem_bytes<64>());
        prepare(reinterpret_cast<const void*>(grouped_tokens_kernel<160>), tokens_smem_bytes<160>());
        prepare(reinterpret_cast<const void*>(grouped_rows_kernel), sizeof(RowsSmem) + 1024);
        int sms = 0;
        if (k.err == cudaSuccess) k.err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        k.pairs = static_cast<uint32_t>(sms) / 2u < kGroupedMaxPairs ? static_cast<uint32_t>(sms) / 2u : kGroupedMaxPairs;
    }
    return k;
}

// Rows of a block of the kernel with tokens on N that the mean number of rows per
// expert calls for, or 0 for the kernel with rows on M. Measured with 32 experts,
// N = 4096, K = 5120, quantizer included (us at 16, 48, 64, 112, 144, 176, 256 rows
// per expert):
//   blocks of 64    124  128  159  215  305  309  447
//   blocks of 160   134  137  140  185  209  260  341
//   rows on M       181  191  192  197  205  210  291
// Below the first crossing the weight stream from DRAM binds both; above the last
// the full 256-row tiles do more per K block. At 146 rows in a long run, where the
// chip's power limit sets the clock, blocks of 160 take 451 us and rows on M 467.
// The mean is all that the host knows: it counts dropped slots and empty experts. Rows
// that gather in a few experts (of 64; blocks of 64, of 160, rows on M, us): 512 in 2
// experts 36, 32, 31, in 8 39, 44, 55, of which the first is taken; 4096 in 16 experts
// 207, 174, 116, the second.
uint32_t tokens_block(uint32_t total, uint32_t experts) {
    return total <= 56u * experts ? 64u : total <= 152u * experts ? 160u : 0u;
}

// The bf16 output [rows, cols] written in [32 x 64] blocks with the 128-byte swizzle.
bool make_out_map(CUtensorMap* map, void* base, uint64_t cols, uint64_t rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[2] = {cols, rows};
    cuuint64_t strides[1] = {cols * 2};
    cuuint32_t box[2] = {kOutCols, 32};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

size_t grouped_partial_bytes(uint32_t total, uint32_t experts) {
    const uint32_t block = tokens_block(total, experts);
    const size_t per_cta = block ? BW * block : BM * BN;
    return static_cast<size_t>(kGroupedMaxPairs) * 2 * 2 * per_cta * sizeof(float);
}

cudaError_t launch_grouped(const GroupedLaunch& L, cudaStream_t stream) {
    const Setup& ks = setup_for_device();
    if (ks.err != cudaSuccess) return ks.err;
    const uint32_t block = tokens_block(L.total, L.experts);
    const bool few = block != 0;
    const uint32_t pad = (L.total + 15u) / 16u * 16u;
    GroupedShape sh;
    sh.total = L.total;
    sh.experts = L.experts;
    sh.N = L.n;
    sh.G = L.k / BK;
    sh.num_n = (L.n + BW_PAIR - 1) / BW_PAIR;
    sh.total_pad = pad;
    sh.w_per_row = L.w_per_row ? 1u : 0u;
    sh.no_copies = L.diag_budget != 0 ? 1u : 0u;
    sh.budget = L.diag_budget != 0 ? L.diag_budget : kWaitBudgetCycles;
    CUtensorMap tw, tt, tx;  // weights, rows, and the scales (tokens kernel) or the output (rows kernel)
    if (!make_map(&tw, L.wq, L.k, static_cast<uint64_t>(L.experts) * L.n, few ? BW : BN_CTA / 2) ||
        !make_map(&tt, L.q, L.k, L.total, few ? 16u : BM) ||
        !(few ? make_scale_map(&tx, L.s_k, pad, sh.G, block + 4u) : make_out_map(&tx, L.y, L.n, L.total)))
        return cudaErrorInvalidValue;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * ks.pairs, 1, 1);
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = block == 64 ? tokens_smem_bytes<64>() : few ? tokens_smem_bytes<160>() : sizeof(RowsSmem) + 1024;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e =
        few ? cudaLaunchKernelEx(&cfg, block == 64 ? grouped_tokens_kernel<64> : grouped_tokens_kernel<160>, tw, tt, tx, L.w_scale, L.offsets, static_cast<uint16_t*>(L.y),
                                 L.partial, L.counters, sh)
            : cudaLaunchKernelEx(&cfg, grouped_rows_kernel, tt, tw, tx, L.s_k, L.w_scale, L.offsets,
                                 static_cast<uint16_t*>(L.y), L.partial, L.counters, sh);
    note_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_quant_rows(const QuantRowsLaunch& L, cudaStream_t stream) {
    const uint32_t G = L.k / 128u, groups = L.total * G;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((groups + 32u * kQuantGroups - 1) / (32u * kQuantGroups), 1, 1);
    cfg.blockDim = dim3(256, 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, quant_rows_kernel, static_cast<const uint16_t*>(L.x), L.rows,
                                             static_cast<uint8_t*>(L.q), L.s_k, L.counters, L.num_counters, L.tokens,
                                             groups, G, (L.total + 15u) / 16u * 16u);
    note_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t read_clear_grouped_error(uint32_t* code, cudaStream_t stream) {
    cudaError_t e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return e;
    uint32_t zero = 0;
    e = cudaMemcpyFromSymbol(code, g_grouped_error, sizeof(uint32_t));
    if (e != cudaSuccess) return e;
    if (*code) e = cudaMemcpyToSymbol(g_grouped_error, &zero, sizeof(uint32_t));
    return e;
}

}  // namespace fp8q
