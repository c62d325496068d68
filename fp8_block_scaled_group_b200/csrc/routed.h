// Host-side declarations of the routed operators (routing plan, grouped
// projection, mixture-of-experts FFN, adapters).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fp8q {

constexpr uint32_t kMaxExperts = 384;

// --------------------------------------------------------- routing plan --

struct RouteLaunch {
    const int32_t* ids;  // [slots]
    int32_t* offsets;    // [experts + 1]
    int32_t* rows;       // [slots]
    int32_t* pos;        // [slots]
    uint32_t slots, topk, experts;
};

cudaError_t launch_moe_route(const RouteLaunch& L, cudaStream_t stream);

// -------------------------------------------------- grouped projection --

// Grouped rows quantized per 128 columns: e4m3 codes [total, k] and K-major
// scales [k/128, ceil16(total)], and `counters` words set to zero for the
// grouped projections that follow.
struct QuantRowsLaunch {
    const void* x;        // bf16 [tokens, k]
    const int32_t* rows;  // [total] row of x of each grouped row, or null: row i
    void* q;
    float* s_k;
    uint32_t* counters;
    uint32_t tokens, total, k, num_counters;
};

cudaError_t launch_quant_rows(const QuantRowsLaunch& L, cudaStream_t stream);

struct GroupedLaunch {
    const void* q;           // e4m3 [total, k]
    const float* s_k;        // fp32 [k/128, ceil16(total)]
    const int32_t* offsets;  // [experts + 1]
    const void* wq;          // e4m3 [experts, n, k]
    const float* w_scale;
    void* y;                 // bf16 [total, n]
    float* partial;          // grouped_partial_bytes()
    uint32_t* counters;      // kGroupedCounters words, zero
    uint32_t total, experts, n, k;
    bool w_per_row;
    // Timeout diagnostics only (0 in normal use): the kernel's producer
    // issues no copies and each wait is bounded by this many clocks.
    long long diag_budget = 0;
};

// Split-K bookkeeping of one grouped projection.
constexpr uint32_t kGroupedMaxPairs = 74;
constexpr uint32_t kGroupedSplitWaves = 4;  // tiles per pair below which the K blocks are split evenly
constexpr uint32_t kGroupedCounters = kGroupedMaxPairs * kGroupedSplitWaves * 16;

size_t grouped_partial_bytes(uint32_t total, uint32_t experts);
cudaError_t launch_grouped(const GroupedLaunch& L, cudaStream_t stream);
// ---------------------------------------------- mixture-of-experts FFN --

// Tokens quantized into the grouped rows of their slots: e4m3 codes [slots, k],
// K-major scales [k/128, ceil16(slots)]; `counters` words are set to zero.
struct MoeQuantLaunch {
    const void* x;       // bf16 [tokens, k]
    const int32_t* pos;  // [tokens, topk]
    void* q;
    float* s_k;
    uint32_t* counters;
    uint32_t tokens, topk, k, num_counters;
};

cudaError_t launch_moe_quant(const MoeQuantLaunch& L, cudaStream_t stream);

// SiLU(gate) * up of the first *kept grouped rows, quantized.
struct MoeSiluLaunch {
    const void* gate_up;  // bf16 [slots, 2i]
    const int32_t* kept;  // device: rows in use
    void* q;
    float* s_k;  // fp32 [i/128, ceil16(slots)]
    uint32_t slots, i;
};

cudaError_t launch_moe_silu_quant(const MoeSiluLaunch& L, cudaStream_t stream);

struct CombineLaunch {
    const void* s;       // bf16 [tokens * topk, d] in grouped order
    const int32_t* pos;  // [tokens, topk]
    const float* p;      // [tokens, topk]
    void* y;             // bf16 [tokens, d]
    uint32_t tokens, topk, d;
};

cudaError_t launch_moe_combine(const CombineLaunch& L, cudaStream_t stream);

// ------------------------------------------------------------ adapters --

// Quantizes x (codes and K-major scales, as the activation quantizer) and
// forms v = scaling[a] A_a x of the rows that have an adapter: fp32 for the decode
// kernel (v_fp32; always for m <= kDecodeMaxTokens), else two bf16 parts, and `lists` too.
struct LoraPrepLaunch {
    const void* x;
    const int32_t* ids;
    const void* a;  // bf16 [adapters, rank, k]
    const void* b;  // bf16 [adapters, n, rank]: brought to L2 for the projection
    const float* scaling;
    void* q;
    float* s_k;
    void* v;
    int32_t* lists;
    uint32_t m, n, k, mp, adapters, rank;
    bool v_fp32;
};

cudaError_t launch_lora_prep(const LoraPrepLaunch& L, uint32_t sms, cudaStream_t stream);

cudaError_t read_clear_grouped_error(uint32_t* code, cudaStream_t stream);

}  // namespace fp8q
