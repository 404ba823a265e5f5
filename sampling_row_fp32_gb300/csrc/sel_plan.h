// sel_plan.h -- host-side helpers: sizes, the device's SM count, and the
// workspace layout shared by the operations.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "sel.h"

namespace sel {

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

inline uint32_t ceil_div(uint64_t a, uint64_t b) {
    return static_cast<uint32_t>((a + b - 1) / b);
}

// Multiprocessor count of the current device (0 if it cannot be queried).
int device_sms();

// Lets kernel K use `bytes` of dynamic shared memory: asked of the driver once
// for each device.
template <auto K>
inline bool dynamic_smem_once(size_t bytes) {
    static std::atomic<uint64_t> done{0};  // a bit a device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return true;
    if (cudaFuncSetAttribute(K, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)) != cudaSuccess)
        return false;
    done.fetch_or(bit, std::memory_order_relaxed);
    return true;
}

// Workspace bytes of each operation (0 when none is needed).
size_t argmax_ws_bytes(uint32_t rows, uint32_t V);
// sel_argmax's main launch alone, folding each row's (max, lowest argmax id)
// key into slots[row] (zero beforehand; all ones for a nonfinite row)
sel_status argmax_into_slots(const float* d_logits, uint32_t rows, uint32_t V, unsigned long long* slots,
                             cudaStream_t stream);
size_t topk_ws_bytes(uint32_t rows, uint32_t V, uint32_t k);
size_t spec_ws_bytes(uint32_t S, uint32_t V, uint32_t K);
size_t spec_diag_ws_bytes(uint32_t S, uint32_t V, uint32_t K);
size_t spec_sampler_ws_bytes(uint32_t rows_t, uint32_t V, uint32_t top_k);
size_t shard_draw_ws_bytes(uint32_t rows, uint32_t V);
size_t spec_shard_draw_ws_bytes(uint32_t S, uint32_t V);
size_t head_loss_ws_bytes(uint32_t rows, uint32_t V, uint32_t H);
size_t head_loss_grad_ws_bytes(uint32_t rows, uint32_t V, uint32_t H);

// Candidates of full-row sampling (sel_sample with top_k = 0).
constexpr uint32_t kFullRowCandidates = 64;

// Workspace: a 256-byte header (word 0: error flags the kernels raise), a
// per-row arrival counter array, then the per-op payload.
constexpr size_t kWsHeaderBytes = 256;
inline size_t ws_counters_bytes(uint32_t rows) { return align_up(static_cast<size_t>(rows) * 4u, 256); }

}  // namespace sel
