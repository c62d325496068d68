// C ABI of the routed operators: argument checks, workspace layouts and the
// launch sequence of each call. Declarations and contracts: include/fp8q.h.
#include "fp8q.h"
#include "internal.h"
#include "ptx.cuh"
#include "routed.h"

using namespace fp8q;

namespace {

constexpr uint32_t kGroup = 128;
constexpr uint64_t kLimit = 1ull << 31;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

size_t round_up(size_t v) { return (v + 255) / 256 * 256; }

fp8q_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return FP8Q_OK;
    cudaGetLastError();
    return FP8Q_ERR_CUDA;
}

// FP8Q_OK on a device of compute capability 10.0.
fp8q_status check_device() {
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess) {
        cudaGetLastError();
        return FP8Q_ERR_CUDA;
    }
    return major == 10 && minor == 0 ? FP8Q_OK : FP8Q_ERR_UNSUPPORTED_DEVICE;
}

bool bad_dim(uint32_t v) { return v == 0 || v % kGroup; }
bool bad_format(int32_t f) { return f != FP8Q_WEIGHT_BLOCK128 && f != FP8Q_WEIGHT_PER_ROW; }

fp8q_status check_route_sizes(uint32_t tokens, uint32_t topk, uint32_t experts) {
    if (experts == 0 || experts > FP8Q_MAX_EXPERTS || topk == 0 || topk > FP8Q_MAX_TOPK) return FP8Q_ERR_SHAPE;
    return static_cast<uint64_t>(tokens) * topk < kLimit / kGroup ? FP8Q_OK : FP8Q_ERR_SHAPE;
}

fp8q_status check_grouped_sizes(uint32_t tokens, uint32_t total, uint32_t experts, uint32_t n, uint32_t k) {
    if (bad_dim(n) || bad_dim(k) || experts == 0 || experts > FP8Q_MAX_EXPERTS) return FP8Q_ERR_SHAPE;
    if (static_cast<uint64_t>(tokens) * k >= kLimit || static_cast<uint64_t>(total) * k >= kLimit ||
        static_cast<uint64_t>(total) * n >= kLimit ||
        static_cast<uint64_t>(n) * k >= kLimit || static_cast<uint64_t>(experts) * n >= kLimit)
        return FP8Q_ERR_SHAPE;
    return FP8Q_OK;
}

// The plan and both projections of the FFN.
fp8q_status check_moe_sizes(uint32_t tokens, uint32_t topk, uint32_t experts, uint32_t d, uint32_t i) {
    fp8q_status st = check_route_sizes(tokens, topk, experts);
    if (st != FP8Q_OK) return st;
    if (i >= kLimit / 2) return FP8Q_ERR_SHAPE;
    const uint32_t slots = tokens * topk;
    if ((st = check_grouped_sizes(tokens, slots, experts, 2 * i, d)) != FP8Q_OK) return st;
    return check_grouped_sizes(slots, slots, experts, d, i);
}

// Offsets of the grouped projection's workspace: codes, scales, counters, partials, end.
void grouped_layout(uint32_t total, uint32_t experts, uint32_t k, size_t (&off)[5]) {
    off[0] = 0;
    off[1] = off[0] + round_up(static_cast<size_t>(total) * k);
    off[2] = off[1] + round_up(static_cast<size_t>(fp8q_m_pad(total)) * (k / kGroup) * sizeof(float));
    off[3] = off[2] + round_up(kGroupedCounters * sizeof(uint32_t));
    off[4] = off[3] + round_up(grouped_partial_bytes(total, experts));
}

// Offsets of the FFN's workspace.
struct MoeLayout {
    size_t offsets, rows, pos, q_x, s_x, gate_up, q_h, s_h, out, counters, partial, total;
};

MoeLayout moe_layout(uint32_t tokens, uint32_t topk, uint32_t experts, uint32_t d, uint32_t i) {
    const size_t slots = static_cast<size_t>(tokens) * topk;
    MoeLayout l;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += round_up(bytes);
        return here;
    };
    l.offsets = take((experts + 1) * sizeof(int32_t));
    l.rows = take(slots * sizeof(int32_t));
    l.pos = take(slots * sizeof(int32_t));
    const size_t pad = (slots + 15) / 16 * 16;
    l.q_x = take(slots * d);
    l.s_x = take(pad * (d / kGroup) * sizeof(float));
    l.gate_up = take(slots * 2 * i * sizeof(uint16_t));
    l.q_h = take(slots * i);
    l.s_h = take(pad * (i / kGroup) * sizeof(float));
    l.out = take(slots * d * sizeof(uint16_t));
    l.counters = take(2 * kGroupedCounters * sizeof(uint32_t));
    l.partial = take(grouped_partial_bytes(static_cast<uint32_t>(slots), experts));
    l.total = at;
    return l;
}

fp8q_status check_lora_sizes(uint32_t m, uint32_t n, uint32_t k, uint32_t adapters, uint32_t rank) {
    if (bad_dim(n) || bad_dim(k) || adapters == 0 || rank == 0 || rank % 8 || rank > FP8Q_MAX_RANK) return FP8Q_ERR_SHAPE;
    if (static_cast<uint64_t>(m) * k >= kLimit || static_cast<uint64_t>(m) * n >= kLimit ||
        static_cast<uint64_t>(n) * k >= kLimit || static_cast<uint64_t>(adapters) * n >= kLimit)
        return FP8Q_ERR_SHAPE;
    return FP8Q_OK;
}

// Whether the decode kernel runs the projection with adapters, 64 rows at a time:
// always for a decode batch, and up to 256 rows while its second sum, m n rank
// products on the CUDA cores, is small. The pair kernel multiplies every adapter of
// 256 rows with all of them, 32 of the rank at a time. How many adapters the rows use
// decides as well, but only the device knows it. Decode against pair kernel, us at
// N = 6144, K = 5120: 128 rows, one adapter of rank 16, 28 and 32; 8 of them, 36 and 42;
// 64, 65 and 98; one of rank 64, 43 and 33; 8, 77 and 51; 64, 122 and 135; 256 rows, 8
// adapters of rank 16, 57 and 44; 64, 104 and 120; at N = 1792, K = 4224, 8, 25 and 34.
bool lora_decode(uint32_t m, uint32_t n, uint32_t rank) {
    if (m <= kDecodeMaxTokens) return true;
    return m <= 256 && static_cast<uint64_t>(m) * n <= 1200000u && static_cast<uint64_t>(rank) * n <= 200000u;
}

// Offsets of the adapters' workspace: codes, K-major scales, v (room for either form), lists of adapters, end.
void lora_layout(uint32_t m, uint32_t k, uint32_t rank, size_t (&off)[5]) {
    off[0] = 0;
    off[1] = off[0] + round_up(static_cast<size_t>(m) * k);
    off[2] = off[1] + round_up(static_cast<size_t>(fp8q_m_pad(m)) * (k / kGroup) * sizeof(float));
    off[3] = off[2] + round_up(static_cast<size_t>(m) * v_parts(rank) * sizeof(uint16_t));
    off[4] = off[3] + round_up((static_cast<size_t>(m) + 255) / 256 * kAdapterList * sizeof(int32_t));
}

fp8q_status check_workspace(const void* workspace, size_t bytes, size_t need) {
    return (reinterpret_cast<uintptr_t>(workspace) & 255u) == 0 && bytes >= need ? FP8Q_OK : FP8Q_ERR_WORKSPACE;
}

// fp8q_grouped_linear; `diag_budget` as in GroupedLaunch.
fp8q_status grouped_linear(const void* x, const int32_t* offsets, const int32_t* rows, const void* wq,
                           const float* w_scale, int32_t weight_format, void* y, void* workspace,
                           size_t workspace_bytes, uint32_t tokens, uint32_t total_rows, uint32_t experts,
                           uint32_t n, uint32_t k, long long diag_budget, void* stream) {
    if (bad_format(weight_format)) return FP8Q_ERR_ARG;
    fp8q_status st = check_grouped_sizes(tokens, total_rows, experts, n, k);
    if (st != FP8Q_OK) return st;
    if (!rows && tokens != total_rows) return FP8Q_ERR_SHAPE;
    if (tokens == 0 || total_rows == 0) return FP8Q_OK;
    if (!x || !offsets || !wq || !w_scale || !y || !workspace) return FP8Q_ERR_NULL;
    if (!aligned16(x) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(y) || !aligned4(offsets) || !aligned4(rows))
        return FP8Q_ERR_ALIGN;
    size_t off[5];
    grouped_layout(total_rows, experts, k, off);
    if ((st = check_workspace(workspace, workspace_bytes, off[4])) != FP8Q_OK) return st;
    if ((st = check_device()) != FP8Q_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    float* s_k = reinterpret_cast<float*>(ws + off[1]);
    uint32_t* counters = reinterpret_cast<uint32_t*>(ws + off[2]);
    QuantRowsLaunch quant{x, rows, ws, s_k, counters, tokens, total_rows, k, kGroupedCounters};
    if ((st = from_cuda(launch_quant_rows(quant, s))) != FP8Q_OK) return st;
    GroupedLaunch L{ws, s_k, offsets, wq, w_scale, y, reinterpret_cast<float*>(ws + off[3]), counters,
                    total_rows, experts, n, k, weight_format == FP8Q_WEIGHT_PER_ROW, diag_budget};
    return from_cuda(launch_grouped(L, s));
}

}  // namespace

extern "C" {

fp8q_status fp8q_moe_route(const int32_t* topk_ids, int32_t* offsets, int32_t* rows, int32_t* pos, uint32_t tokens,
                           uint32_t topk, uint32_t experts, void* stream) {
    fp8q_status st = check_route_sizes(tokens, topk, experts);
    if (st != FP8Q_OK) return st;
    if (!offsets) return FP8Q_ERR_NULL;
    if (tokens != 0 && (!topk_ids || !rows || !pos)) return FP8Q_ERR_NULL;
    if (!aligned4(topk_ids) || !aligned4(offsets) || !aligned4(rows) || !aligned4(pos)) return FP8Q_ERR_ALIGN;
    if ((st = check_device()) != FP8Q_OK) return st;
    RouteLaunch L{topk_ids, offsets, rows, pos, tokens * topk, topk, experts};
    return from_cuda(launch_moe_route(L, static_cast<cudaStream_t>(stream)));
}

size_t fp8q_grouped_linear_workspace_bytes(uint32_t tokens, uint32_t total_rows, uint32_t experts, uint32_t n,
                                           uint32_t k) {
    if (check_grouped_sizes(tokens, total_rows, experts, n, k) != FP8Q_OK) return 0;
    size_t off[5];
    grouped_layout(total_rows, experts, k, off);
    return off[4];
}

fp8q_status fp8q_grouped_linear(const void* x, const int32_t* offsets, const int32_t* rows, const void* wq,
                                const float* w_scale, int32_t weight_format, void* y, void* workspace,
                                size_t workspace_bytes, uint32_t tokens, uint32_t total_rows, uint32_t experts,
                                uint32_t n, uint32_t k, void* stream) {
    return grouped_linear(x, offsets, rows, wq, w_scale, weight_format, y, workspace, workspace_bytes, tokens, total_rows,
                          experts, n, k, 0, stream);
}

fp8q_status fp8q_diag_stalled_grouped_linear(const void* x, const int32_t* offsets, const int32_t* rows, const void* wq,
                                             const float* w_scale, int32_t weight_format, void* y, void* workspace,
                                             size_t workspace_bytes, uint32_t tokens, uint32_t total_rows,
                                             uint32_t experts, uint32_t n, uint32_t k, uint64_t wait_budget_cycles,
                                             void* stream) {
    if (wait_budget_cycles == 0 || wait_budget_cycles > static_cast<uint64_t>(kWaitBudgetCycles)) return FP8Q_ERR_ARG;
    return grouped_linear(x, offsets, rows, wq, w_scale, weight_format, y, workspace, workspace_bytes, tokens, total_rows,
                          experts, n, k, static_cast<long long>(wait_budget_cycles), stream);
}

size_t fp8q_moe_ffn_workspace_bytes(uint32_t tokens, uint32_t topk, uint32_t experts, uint32_t d, uint32_t i) {
    if (check_moe_sizes(tokens, topk, experts, d, i) != FP8Q_OK) return 0;
    return moe_layout(tokens, topk, experts, d, i).total;
}

fp8q_status fp8q_moe_ffn(const void* x, const int32_t* topk_ids, const float* topk_weights, const void* w_gate_up,
                         const float* w_gate_up_scale, const void* w_down, const float* w_down_scale,
                         int32_t weight_format, void* y, void* workspace, size_t workspace_bytes, uint32_t tokens,
                         uint32_t topk, uint32_t experts, uint32_t d, uint32_t i, void* stream) {
    if (bad_format(weight_format)) return FP8Q_ERR_ARG;
    fp8q_status st = check_moe_sizes(tokens, topk, experts, d, i);
    if (st != FP8Q_OK) return st;
    const uint32_t slots = tokens * topk;
    if (tokens == 0) return FP8Q_OK;
    if (!x || !topk_ids || !topk_weights || !w_gate_up || !w_gate_up_scale || !w_down || !w_down_scale || !y || !workspace)
        return FP8Q_ERR_NULL;
    if (!aligned16(x) || !aligned16(w_gate_up) || !aligned16(w_gate_up_scale) || !aligned16(w_down) ||
        !aligned16(w_down_scale) || !aligned16(y) || !aligned4(topk_ids) || !aligned4(topk_weights))
        return FP8Q_ERR_ALIGN;
    const MoeLayout l = moe_layout(tokens, topk, experts, d, i);
    if ((st = check_workspace(workspace, workspace_bytes, l.total)) != FP8Q_OK) return st;
    if ((st = check_device()) != FP8Q_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    int32_t* offsets = reinterpret_cast<int32_t*>(ws + l.offsets);
    int32_t* rows = reinterpret_cast<int32_t*>(ws + l.rows);
    int32_t* pos = reinterpret_cast<int32_t*>(ws + l.pos);
    float* s_x = reinterpret_cast<float*>(ws + l.s_x);
    uint16_t* gu = reinterpret_cast<uint16_t*>(ws + l.gate_up);
    float* s_h = reinterpret_cast<float*>(ws + l.s_h);
    uint32_t* counters = reinterpret_cast<uint32_t*>(ws + l.counters);
    float* partial = reinterpret_cast<float*>(ws + l.partial);
    const bool per_row = weight_format == FP8Q_WEIGHT_PER_ROW;
    // Each launch is the programmatic dependent of the one before it and
    // waits for it before reading or writing global memory.
    RouteLaunch route{topk_ids, offsets, rows, pos, slots, topk, experts};
    if ((st = from_cuda(launch_moe_route(route, s))) != FP8Q_OK) return st;
    MoeQuantLaunch quant{x, pos, ws + l.q_x, s_x, counters, tokens, topk, d, 2 * kGroupedCounters};
    if ((st = from_cuda(launch_moe_quant(quant, s))) != FP8Q_OK) return st;
    GroupedLaunch gate_up{ws + l.q_x, s_x, offsets, w_gate_up, w_gate_up_scale, gu, partial, counters,
                          slots, experts, 2 * i, d, per_row};
    if ((st = from_cuda(launch_grouped(gate_up, s))) != FP8Q_OK) return st;
    MoeSiluLaunch act{gu, offsets + experts, ws + l.q_h, s_h, slots, i};
    if ((st = from_cuda(launch_moe_silu_quant(act, s))) != FP8Q_OK) return st;
    GroupedLaunch down{ws + l.q_h, s_h, offsets, w_down, w_down_scale, ws + l.out, partial,
                       counters + kGroupedCounters, slots, experts, d, i, per_row};
    if ((st = from_cuda(launch_grouped(down, s))) != FP8Q_OK) return st;
    CombineLaunch combine{ws + l.out, pos, topk_weights, y, tokens, topk, d};
    return from_cuda(launch_moe_combine(combine, s));
}

size_t fp8q_lora_linear_workspace_bytes(uint32_t m, uint32_t n, uint32_t k, uint32_t adapters, uint32_t rank) {
    if (check_lora_sizes(m, n, k, adapters, rank) != FP8Q_OK) return 0;
    size_t off[5];
    lora_layout(m, k, rank, off);
    return off[4];
}

fp8q_status fp8q_lora_linear(const void* x, const void* wq, const float* w_scale, int32_t weight_format,
                             const int32_t* adapter_ids, const void* lora_a, const void* lora_b, const float* scaling,
                             void* y, void* workspace, size_t workspace_bytes, uint32_t m, uint32_t n, uint32_t k,
                             uint32_t adapters, uint32_t rank, void* stream) {
    if (bad_format(weight_format)) return FP8Q_ERR_ARG;
    fp8q_status st = check_lora_sizes(m, n, k, adapters, rank);
    if (st != FP8Q_OK) return st;
    if (m == 0) return FP8Q_OK;
    if (!x || !wq || !w_scale || !adapter_ids || !lora_a || !lora_b || !scaling || !y || !workspace) return FP8Q_ERR_NULL;
    if (!aligned16(x) || !aligned16(wq) || !aligned16(w_scale) || !aligned16(lora_a) || !aligned16(lora_b) ||
        !aligned16(y) || !aligned4(adapter_ids) || !aligned4(scaling))
        return FP8Q_ERR_ALIGN;
    size_t off[5];
    lora_layout(m, k, rank, off);
    if ((st = check_workspace(workspace, workspace_bytes, off[4])) != FP8Q_OK) return st;
    if ((st = check_device()) != FP8Q_OK) return st;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    float* s_k = reinterpret_cast<float*>(ws + off[1]);
    int32_t* lists = reinterpret_cast<int32_t*>(ws + off[3]);
    const bool decode = lora_decode(m, n, rank);
    LoraPrepLaunch prep{x, adapter_ids, lora_a, lora_b, scaling, ws, s_k, ws + off[2], decode ? nullptr : lists, m, n, k, fp8q_m_pad(m), adapters, rank, decode};
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return from_cuda(cudaErrorInvalidDevice);
    if ((st = from_cuda(launch_lora_prep(prep, static_cast<uint32_t>(sms), s))) != FP8Q_OK) return st;
    LoraOperands lora{adapter_ids, lists, ws + off[2], lora_b, adapters, rank, decode};
    GemmLaunch L{ws, s_k, wq, w_scale, y, m, n, k, fp8q_m_pad(m), true, weight_format == FP8Q_WEIGHT_PER_ROW};
    L.lora = &lora;
    return from_cuda(launch_gemm(L, s));
}

}  // extern "C"
