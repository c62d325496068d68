// What the two grouped projection kernels share: the experts' groups as blocks
// of rows, the list of pieces of work, and the joining of partial sums.
#pragma once

#include <cstdint>

#include "ptx.cuh"
#include "routed.h"

namespace fp8q {

constexpr uint32_t kGroupedThreads = 384;
constexpr uint32_t kPieceMin = 4;  // K blocks of a split piece, at least
// K blocks per pair that idling in the last round of whole tiles may cost before the
// K range is split: parking and joining partial sums costs about that much. With 8
// experts' weights for one row each (N = 4096, K = 5120: 11 K blocks idle) whole tiles
// take 35 us and split ones 41; at K = 17408 (59 idle) 71 and 59.
constexpr uint32_t kSplitCost = 32;

struct GroupedShape {
    uint32_t total, experts, N, G;
    uint32_t num_n;      // 256-column weight tiles per expert
    uint32_t total_pad;  // row extent of the K-major scales
    uint32_t w_per_row;
    uint32_t no_copies;  // timeout diagnostics: the producer issues no copies
    long long budget;    // clock budget of every wait
};

// The groups, in shared memory.
struct Experts {
    uint32_t warp_sum[kGroupedThreads / 32];
    int32_t begin[kMaxExperts];       // first grouped row of each expert
    uint32_t count[kMaxExperts];      // its rows
    uint32_t block[kMaxExperts + 1];  // row blocks of the experts before it
};

// Fills `ex`; all threads of the CTA call it. Offsets outside [0, total] or out
// of order give empty or clipped groups, never an access out of bounds. A
// thread takes kPer neighbouring experts. They are read from L2: this grid may
// have started while the one before it ran.
template <uint32_t kBlock>
__device__ __forceinline__ void list_experts(Experts& ex, const int32_t* __restrict__ offsets, const GroupedShape& sh) {
    constexpr uint32_t kPer = (kMaxExperts + kGroupedThreads) / kGroupedThreads;  // covers kMaxExperts + 1 entries
    const uint32_t warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t mine[kPer], sum = 0;
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) {
        const uint32_t e = threadIdx.x * kPer + j;
        mine[j] = sum;
        if (e < sh.experts) {
            const int32_t cap = static_cast<int32_t>(sh.total);
            const int32_t a = min(max(__ldcg(offsets + e), 0), cap);
            const int32_t b = min(max(__ldcg(offsets + e + 1), 0), cap);
            const uint32_t n = b > a ? static_cast<uint32_t>(b - a) : 0u;
            ex.begin[e] = a;
            ex.count[e] = n;
            sum += (n + kBlock - 1) / kBlock;
        }
    }
    uint32_t incl = sum;
#pragma unroll
    for (uint32_t o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) ex.warp_sum[warp] = incl;
    __syncthreads();
    uint32_t before = incl - sum;
    for (uint32_t v = 0; v < warp; ++v) before += ex.warp_sum[v];
#pragma unroll
    for (uint32_t j = 0; j < kPer; ++j) {
        const uint32_t e = threadIdx.x * kPer + j;
        if (e <= sh.experts) ex.block[e] = before + mine[j];
    }
}

// One piece of work: K blocks kb0..kb1 of a tile.
struct Piece {
    uint32_t tile, expert, n0;   // n0: first weight row of the pair's tile
    uint32_t row0, rows;         // grouped rows of the row block
    uint32_t kb0, kb1;
};

// The pieces of this pair, in order. Every role of both CTAs walks the same
// list. A block is kBlock rows of an expert; kEven: an expert's blocks are made
// equally long instead of all but the last being full.
template <uint32_t kBlock, bool kEven>
struct Walk {
    const Experts& sm;
    const GroupedShape& sh;
    uint32_t pair, pairs, tiles;
    bool split;
    uint32_t expert = 0;
    uint32_t next = 0;             // the next whole tile
    // Split walk: this pair's piece of the line. The parts of tiles at its two ends
    // come first, so that what joins them is done while the whole tiles stream.
    uint32_t unit = 0, unit_end = 0, head = 0, tail = 0, next_end = 0;

    __device__ __forceinline__ Walk(const Experts& s, const GroupedShape& h, uint32_t p, uint32_t ps)
        : sm(s), sh(h), pair(p), pairs(ps) {
        tiles = sm.block[sh.experts] * sh.num_n;
        // Whole tiles leave this many K blocks x pairs of the last round idle.
        const uint32_t idle = ((tiles + pairs - 1) / pairs * pairs - tiles) * sh.G;
        split = tiles < kGroupedSplitWaves * pairs && idle > kSplitCost * pairs;
        if (split) {
            // At least kPieceMin K blocks a pair; the pairs left over idle.
            const uint32_t most = (tiles * sh.G + kPieceMin - 1) / kPieceMin;
            pairs = pairs < most ? pairs : most;
            if (p < pairs) {
                unit = bound(p);
                unit_end = bound(p + 1);
                next = (unit + sh.G - 1) / sh.G;
                next_end = unit_end / sh.G;
                head = unit < next * sh.G ? 1u : 0u;  // the piece begins inside a tile
                tail = unit_end > next_end * sh.G && next_end >= next ? 1u : 0u;  // it ends inside another
            }
        } else {
            next = p;
        }
    }

    // First K block of pair p's piece of the line: the even cut, moved to a
    // tile's edge when that is a few K blocks away.
    __device__ __forceinline__ uint32_t bound(uint32_t p) const {
        const uint32_t u = static_cast<uint32_t>(static_cast<uint64_t>(tiles) * sh.G * p / pairs);
        const uint32_t r = u % sh.G;
        const uint32_t near = sh.G / 16u;
        if (r <= near) return u - r;
        if (sh.G - r <= near) return u + sh.G - r;
        return u;
    }

    // The pair whose piece holds K block u of the line.
    __device__ __forceinline__ uint32_t owner(uint32_t u) const {
        uint32_t p = static_cast<uint32_t>(static_cast<uint64_t>(u) * pairs / (static_cast<uint64_t>(tiles) * sh.G));
        while (p > 0 && bound(p) > u) --p;
        while (p + 1 < pairs && bound(p + 1) <= u) ++p;
        return p;
    }

    // Few instructions where an expert has one block: a warp that does nothing
    // else meanwhile takes four to five clocks for each.
    __device__ __forceinline__ void locate(uint32_t tile, Piece& w) {
        if (tile < sm.block[expert] * sh.num_n) expert = 0;
        if (tile >= sm.block[expert + 1] * sh.num_n) {
            if (++expert, tile >= sm.block[expert + 1] * sh.num_n) {  // binary search above the last expert
                const uint32_t b = tile / sh.num_n;
                uint32_t lo = expert + 1, hi = sh.experts - 1;
                while (lo < hi) {
                    const uint32_t mid = (lo + hi) >> 1;
                    if (b >= sm.block[mid + 1]) lo = mid + 1;
                    else hi = mid;
                }
                expert = lo;
            }
        }
        const uint32_t first = sm.block[expert];
        const uint32_t blocks = sm.block[expert + 1] - first;
        const uint32_t count = sm.count[expert];
        uint32_t tn = tile - first * sh.num_n, at = 0, per = kEven ? count : kBlock;
        if (blocks > 1) {
            const uint32_t local = tn;
            tn = local / blocks;
            if (kEven) per = (count + blocks - 1) / blocks;
            at = (local - tn * blocks) * per;
        }
        w.tile = tile;
        w.expert = expert;
        w.n0 = tn * 256u;
        w.row0 = static_cast<uint32_t>(sm.begin[expert]) + at;
        w.rows = at < count ? (count - at < per ? count - at : per) : 0u;
    }

    __device__ __forceinline__ bool pop(Piece& w) {
        if (split) {
            if (head) {
                head = 0;
                locate(unit / sh.G, w);
                w.kb0 = unit - w.tile * sh.G;
                const uint32_t left = unit_end - unit;
                w.kb1 = w.kb0 + left < sh.G ? w.kb0 + left : sh.G;
                return true;
            }
            if (tail) {
                tail = 0;
                locate(next_end, w);
                w.kb0 = 0;
                w.kb1 = unit_end - next_end * sh.G;
                return true;
            }
            if (next >= next_end) return false;
            locate(next++, w);
            w.kb0 = 0;
            w.kb1 = sh.G;
            return true;
        }
        if (next >= tiles) return false;
        locate(next, w);
        w.kb0 = 0;
        w.kb1 = sh.G;
        next += pairs;
        return true;
    }
};

// Where a role stands in a ring: slot and parity of the phase.
template <uint32_t kSlots>
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void step() {
        if (++slot == kSlots) {
            slot = 0;
            phase ^= 1u;
        }
    }
};

// A split tile's partial sums. Each of the tile's pairs p_first .. p_last has a
// slot per promotion warp of kFloat4 x 32 lanes x 16 bytes: its second one if
// the tile begins in the pair's piece, else its first.
template <uint32_t kFloat4>
struct Partial {
    float4* slots;
    uint32_t* counter;
    uint32_t pair, p_first, p_last, rank, warp, lane;

    __device__ __forceinline__ float4* slot(uint32_t p) const {
        return slots + (((static_cast<size_t>(p) * 2u + (p == p_first ? 1u : 0u)) * 2u + rank) * 8u + warp) * (kFloat4 * 32u) + lane;
    }
    __device__ __forceinline__ void put(uint32_t i, float4 v) const { slot(pair)[i * 32u] = v; }

    // After this pair's puts: true in the warp that comes last, which then
    // reads all parts. The order of arrival does not enter the sums.
    __device__ __forceinline__ bool last() const {
        __threadfence();
        __syncwarp();
        uint32_t seen = 0;
        if (lane == 0) seen = atomicAdd(counter, 1u);
        seen = __shfl_sync(0xFFFFFFFFu, seen, 0);
        __threadfence();
        return seen == p_last - p_first;
    }
    // Entries i .. i + kCount - 1 of all parts, added in K order.
    template <uint32_t kCount>
    __device__ __forceinline__ void sum(uint32_t i, float4 (&out)[kCount]) const {
#pragma unroll
        for (uint32_t j = 0; j < kCount; ++j) out[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (uint32_t p = p_first; p <= p_last; ++p) {
            const float4* from = slot(p) + i * 32u;
            float4 n[kCount];
#pragma unroll
            for (uint32_t j = 0; j < kCount; ++j) n[j] = __ldcg(from + j * 32u);
#pragma unroll
            for (uint32_t j = 0; j < kCount; ++j) {
                out[j].x += n[j].x;
                out[j].y += n[j].y;
                out[j].z += n[j].z;
                out[j].w += n[j].w;
            }
        }
    }
};

}  // namespace fp8q
