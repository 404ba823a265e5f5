// sel_head.cu -- logits rows of hidden states through a 4-bit output head.
//
//   L[r][v] = sum_g s[v][g] * sum_{k in g} x[r][k] * (q[v][k] - z[v][g])
//
// x is a 16-bit float and q - z an integer in -15..15, which the same 16-bit
// type holds exactly. So the inner sums run on the tensor cores without
// rounding an operand: per group, D[v][r] = (q - z) . x in fp32 (tcgen05, a
// matrix row per TMEM lane), and the scale is applied to D in fp32 outside.
// Folding s into the operand would round s * (q - z) to 16 bits instead.
//
// A persistent CTA per SM owns a run of matrix rows and walks it in tiles of
// 256 (two subtiles of 128 TMEM lanes), each over all columns. Warp roles:
//   warp 0        copies packed weights and hidden states into a ring of
//                 shared-memory stages of 128 columns (TMA, swizzled)
//   warps 4-11    unpack 64 columns of a row each: two 16-byte loads, nibbles
//                 to the type by placing them in the mantissa of 128 (bf16) or
//                 1024 (f16) and subtracting 128 + z (1024 + z), both exact;
//                 the tile goes to TMEM as the product's A operand
//   warp 1        issues the products (A from TMEM, B = hidden states from
//                 shared memory, D in TMEM, double-buffered by group)
//   warps 12-19   read each group's D, add s * D to fp32 registers, and
//                 write the logits after the last group
// Every wait is bounded; one that runs out makes the CTA's logits NaN.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "sel.h"
#include "sel_common.cuh"
#include "sel_dtype.cuh"
#include "sel_plan.h"
#include "sel_units.cuh"

namespace sel {
namespace {

constexpr int kNT = 640;
constexpr uint32_t kTileV = 256;     // matrix rows a tile
constexpr uint32_t kSubV = 128;      // rows a subtile: TMEM lanes
constexpr uint32_t kBoxV = 64;       // rows a weight copy
constexpr uint32_t kStageK = 128;    // columns a stage
constexpr uint32_t kTileK = 64;      // columns an A buffer
constexpr uint32_t kWBytes = kTileV * kStageK / 2;
constexpr uint32_t kABufs = 4, kDBufs = 2;
constexpr uint32_t kACols = kTileK / 2;  // TMEM columns of an A buffer
constexpr uint32_t kMaxStages = 10;

template <int N>
struct Config {
    static constexpr uint32_t kXAtom = N * 128;  // 64 columns of N hidden rows
    static constexpr uint32_t kStageBytes = kWBytes + 2 * kXAtom;
    static constexpr uint32_t kStages = 212 * 1024 / kStageBytes < kMaxStages ? 212 * 1024 / kStageBytes : kMaxStages;
    static constexpr uint32_t kSmem = kStages * kStageBytes + 1024;
    static constexpr uint32_t kACol = 2 * kDBufs * N;  // A buffers lie behind the D buffers
    static_assert(kACol + 2 * kABufs * kACols <= 512);
};

struct HeadArgs {
    const void* scales;
    const uint8_t* zeros;
    void* out;
    uint64_t ld;
    uint32_t rows, V, H, group;
    uint32_t range;  // matrix rows a CTA
};

// ---------------------------------------------------------------------------
// tensor memory and tensor core primitives
// ---------------------------------------------------------------------------

__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// The barrier completes once every product issued before by this thread has.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
// D (+)= A B^T, A [128][16] in TMEM, B [N][16] in shared memory.
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
        : "memory");
}
// 32 consecutive TMEM columns of each lane of the warp's quarter.
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr));
}
// Waits for the loads before it; the registers pass through, so that no use of
// theirs moves ahead of the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory descriptor of a K-major tile of 128-byte rows with the
// 128-byte swizzle: 8-row atoms 1,024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr) {
    return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (1ull << 16) | (static_cast<uint64_t>(1024 >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}

template <typename T>
struct Unpack;
template <>
struct Unpack<__nv_bfloat16> {
    static constexpr uint32_t kMagic = 0x43004300u;  // 128: the mantissa's last bit is 1
    static constexpr uint32_t kType = 1;
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
};
template <>
struct Unpack<__half> {
    static constexpr uint32_t kMagic = 0x64006400u;  // 1024
    static constexpr uint32_t kType = 0;
    static __device__ __forceinline__ uint32_t sub(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
};

// Eight nibbles to four pairs (columns 2 i, 2 i + 1) of q - z.
template <typename T>
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t zc, uint32_t* r) {
    const uint32_t u = w >> 4;
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
        const uint32_t p = __byte_perm(w, u, i | (i << 4) | ((4 + i) << 8) | ((4 + i) << 12));
        r[i] = Unpack<T>::sub((p & 0x000F000Fu) | Unpack<T>::kMagic, zc);
    }
}

__device__ __forceinline__ void fma2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t s) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(d), "l"(s));
}

struct Ctx {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t a_full[2][kABufs], a_empty[2][kABufs];
    uint64_t d_full[2][kDBufs], d_empty[2][kDBufs];
    uint64_t drain;
    uint32_t tmem;
    uint32_t err;
};

template <typename T, typename O, int N>
__global__ void __launch_bounds__(kNT, 1)
    head_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, HeadArgs a) {
    using C = Config<N>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    __shared__ Ctx c;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    if (tid == 0) {
        for (uint32_t i = 0; i < C::kStages; ++i) {
            mbar_init(&c.full[i], 1);
            mbar_init(&c.empty[i], 8 + 1);  // the unpacking warps and the products
        }
        for (uint32_t s = 0; s < 2; ++s) {
            for (uint32_t i = 0; i < kABufs; ++i) {
                mbar_init(&c.a_full[s][i], 4);
                mbar_init(&c.a_empty[s][i], 1);
            }
            for (uint32_t i = 0; i < kDBufs; ++i) {
                mbar_init(&c.d_full[s][i], 1);
                mbar_init(&c.d_empty[s][i], 4);
            }
        }
        mbar_init(&c.drain, 1);
        c.err = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&c.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = c.tmem;
    pdl_wait();
    pdl_trigger();

    const uint32_t v_begin = blockIdx.x * a.range, v_end = min(a.V, v_begin + a.range);
    const uint32_t blocks = (a.rows + N - 1) / N;  // blocks of hidden rows
    const uint32_t stages = (a.H + kStageK - 1) / kStageK;
    const uint32_t ktiles = (a.H + kTileK - 1) / kTileK;
    const uint32_t groups = a.H / a.group;
    bool ok = true;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t it = 0;
            for (uint32_t vt = v_begin; vt < v_end && ok; vt += kTileV) {
                const uint32_t boxes = (min(kTileV, v_end - vt) + kBoxV - 1) / kBoxV;
                for (uint32_t blk = 0; blk < blocks && ok; ++blk) {
                    for (uint32_t st = 0; st < stages; ++st, ++it) {
                        const uint32_t slot = it % C::kStages;
                        ok = mbar_wait(&c.empty[slot], ((it / C::kStages) & 1) ^ 1);
                        if (!ok) break;
                        unsigned char* dst = ring + slot * C::kStageBytes;
                        const uint32_t atoms = st * kStageK + kTileK < a.H ? 2 : 1;
                        expect_tx(&c.full[slot], boxes * kBoxV * (kStageK / 2) + atoms * C::kXAtom);
                        for (uint32_t b = 0; b < boxes; ++b)
                            tma_2d(dst + b * kBoxV * (kStageK / 2), &map_w, st * (kStageK / 2), vt + b * kBoxV,
                                   &c.full[slot]);
                        for (uint32_t at = 0; at < atoms; ++at)
                            tma_2d(dst + kWBytes + at * C::kXAtom, &map_x, st * kStageK + at * kTileK, blk * N,
                                   &c.full[slot]);
                    }
                }
            }
            // every copy has landed before the CTA may end (on the normal path
            // each wait succeeds at once or as the consumers' did)
            for (uint32_t i = it > C::kStages ? it - C::kStages : 0; i < it; ++i)
                if (!mbar_wait(&c.full[i % C::kStages], (i / C::kStages) & 1)) ok = false;
            if (!ok) c.err = 1;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t idesc = (1u << 4) | (Unpack<T>::kType << 7) | (Unpack<T>::kType << 10) |
                                   (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(kSubV >> 4) << 24);
            uint32_t it = 0, ac[2] = {0, 0}, dc[2] = {0, 0};
            for (uint32_t vt = v_begin; vt < v_end && ok; vt += kTileV) {
                const uint32_t subs = v_end - vt > kSubV ? 2 : 1;
                for (uint32_t blk = 0; blk < blocks && ok; ++blk) {
                    for (uint32_t kt = 0; kt < ktiles && ok; ++kt) {
                        const uint32_t slot = it % C::kStages;
                        if ((kt & 1) == 0) ok = mbar_wait(&c.full[slot], (it / C::kStages) & 1);
                        const uint32_t steps = min(4u, (a.H - kt * kTileK) / 16);
                        const uint64_t b0 =
                            smem_desc(smem_u32(ring + slot * C::kStageBytes + kWBytes + (kt & 1) * C::kXAtom));
#pragma unroll
                        for (uint32_t s = 0; s < 2; ++s) {
                            if (s >= subs || !ok) continue;
                            const uint32_t buf = ac[s] % kABufs;
                            ok = mbar_wait(&c.a_full[s][buf], (ac[s] / kABufs) & 1);
                            if (!ok) continue;
                            tc_fence_after();
                            const uint32_t a0 = tmem + C::kACol + (s * kABufs + buf) * kACols;
                            for (uint32_t j = 0; j < steps; ++j) {
                                const uint32_t k = kt * kTileK + j * 16;
                                const bool first = k % a.group == 0;
                                const uint32_t db = dc[s] % kDBufs;
                                if (first) {
                                    ok = mbar_wait(&c.d_empty[s][db], ((dc[s] / kDBufs) & 1) ^ 1);
                                    if (!ok) break;
                                    tc_fence_after();
                                }
                                tc_mma(tmem + (s * kDBufs + db) * N, a0 + j * 8, b0 + j * 2, idesc, !first);
                                if ((k + 16) % a.group == 0) {
                                    tc_commit(&c.d_full[s][db]);
                                    ++dc[s];
                                }
                            }
                            tc_commit(&c.a_empty[s][buf]);
                            ++ac[s];
                        }
                        if ((kt & 1) || kt + 1 == ktiles) {
                            tc_commit(&c.empty[slot]);
                            ++it;
                        }
                    }
                }
            }
            // no product is in flight when the tensor memory is given back
            tc_commit(&c.drain);
            if (!mbar_wait(&c.drain, 0)) ok = false;
            if (!ok) c.err = 1;
        }
        __syncwarp();
    } else if (warp >= 4 && warp < 12) {
        const uint32_t s = (warp - 4) / 4, quarter = warp & 3;
        const uint32_t row = s * kSubV + quarter * 32 + lane;
        const uint32_t a0 = tmem + (quarter << 21) + C::kACol + s * kABufs * kACols;
        // 16-byte chunk ch of a 64-byte row lies at ch ^ ((row >> 1) & 3)
        const uint32_t w0 = row * 64, sw = (row >> 1) & 3;
        uint32_t it = 0, ac = 0;
        for (uint32_t vt = v_begin; vt < v_end && ok; vt += kTileV) {
            const bool active = s == 0 || v_end - vt > kSubV;
            const uint8_t* z = a.zeros ? a.zeros + static_cast<uint64_t>(min(vt + row, a.V - 1)) * groups : nullptr;
            for (uint32_t blk = 0; blk < blocks && ok; ++blk) {
                for (uint32_t kt = 0; kt < ktiles; ++kt) {
                    const uint32_t slot = it % C::kStages;
                    if ((kt & 1) == 0) ok = __all_sync(kFull, mbar_wait(&c.full[slot], (it / C::kStages) & 1));
                    if (!ok) break;
                    const bool last = (kt & 1) || kt + 1 == ktiles;
                    if (active) {
                        const uint32_t buf = ac % kABufs;
                        const unsigned char* src = ring + slot * C::kStageBytes + w0;
                        const uint32_t ch = (kt & 1) * 2;
                        const uint4 q0 = *reinterpret_cast<const uint4*>(src + ((ch ^ sw) << 4));
                        const uint4 q1 = *reinterpret_cast<const uint4*>(src + (((ch + 1) ^ sw) << 4));
                        uint32_t z0 = 8, z1 = 8;
                        if (z) {
                            const uint32_t g = kt * kTileK / a.group;
                            z0 = z[g] & 15;
                            z1 = a.group == 32 && g + 1 < groups ? z[g + 1] & 15 : z0;
                        }
                        const uint32_t zc0 = Unpack<T>::kMagic | z0 | (z0 << 16), zc1 = Unpack<T>::kMagic | z1 | (z1 << 16);
                        uint32_t r[32];
                        unpack8<T>(q0.x, zc0, r);
                        unpack8<T>(q0.y, zc0, r + 4);
                        unpack8<T>(q0.z, zc0, r + 8);
                        unpack8<T>(q0.w, zc0, r + 12);
                        unpack8<T>(q1.x, zc1, r + 16);
                        unpack8<T>(q1.y, zc1, r + 20);
                        unpack8<T>(q1.z, zc1, r + 24);
                        unpack8<T>(q1.w, zc1, r + 28);
                        ok = __all_sync(kFull, mbar_wait(&c.a_empty[s][buf], ((ac / kABufs) & 1) ^ 1));
                        if (!ok) break;
                        tc_fence_after();
                        tmem_st32(a0 + buf * kACols, r);
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive(&c.a_full[s][buf]);
                        ++ac;
                    }
                    if (last) {
                        __syncwarp();
                        if (lane == 0) arrive(&c.empty[slot]);
                        ++it;
                    }
                }
            }
        }
        if (!ok) c.err = 1;
    } else if (warp >= 12) {
        const uint32_t s = (warp - 12) / 4, quarter = warp & 3;
        const uint32_t row = s * kSubV + quarter * 32 + lane;
        const uint32_t d0 = tmem + (quarter << 21) + s * kDBufs * N;
        uint32_t dc = 0;
        for (uint32_t vt = v_begin; vt < v_end && ok; vt += kTileV) {
            if (s == 1 && v_end - vt <= kSubV) continue;
            const T* sc = static_cast<const T*>(a.scales) + static_cast<uint64_t>(min(vt + row, a.V - 1)) * groups;
            for (uint32_t blk = 0; blk < blocks && ok; ++blk) {
                uint64_t acc[N / 2];
#pragma unroll
                for (int i = 0; i < N / 2; ++i) acc[i] = 0;
                T next = sc[0];
                for (uint32_t g = 0; g < groups; ++g, ++dc) {
                    const uint32_t sf = __float_as_uint(to_f32(next));
                    if (g + 1 < groups) next = sc[g + 1];
                    uint64_t s2;
                    asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "r"(sf));
                    const uint32_t db = dc % kDBufs;
                    ok = __all_sync(kFull, mbar_wait(&c.d_full[s][db], (dc / kDBufs) & 1));
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < N / 16; ++h) {
                        uint32_t d[16];
                        tmem_ld16(d0 + db * N + h * 16, d);
                        tmem_wait_ld(d);
                        if (h == N / 16 - 1) {  // the buffer is read
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) arrive(&c.d_empty[s][db]);
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) fma2(acc[h * 8 + i], d[2 * i], d[2 * i + 1], s2);
                    }
                }
                if (!ok) break;
                if (vt + row < v_end) {
                    O* out = static_cast<O*>(a.out) + static_cast<uint64_t>(blk) * N * a.ld + vt + row;
                    const uint32_t n = min(static_cast<uint32_t>(N), a.rows - blk * N);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const uint32_t bits = static_cast<uint32_t>(acc[i / 2] >> (32 * (i & 1)));
                        if (static_cast<uint32_t>(i) < n) out[static_cast<uint64_t>(i) * a.ld] = from_f32<O>(__uint_as_float(bits));
                    }
                }
            }
        }
        if (!ok) c.err = 1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    if (c.err) {  // a wait ran out: nothing this CTA wrote can be trusted
        for (uint32_t r = 0; r < a.rows; ++r)
            for (uint32_t v = v_begin + tid; v < v_end; v += kNT)
                static_cast<O*>(a.out)[r * a.ld + v] = from_f32<O>(__uint_as_float(0x7FC00000u));
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static const EncodeTiled f = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult r{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            p = nullptr;
        }
        return reinterpret_cast<EncodeTiled>(p);
    }();
    return f;
}

// A row-major matrix [rows][cols] read in boxes of box_cols x box_rows.
bool make_map(CUtensorMap* map, CUtensorMapDataType type, uint32_t elem, const void* base, uint64_t cols, uint64_t rows,
              uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols * elem};
    const cuuint32_t box[2] = {box_cols, box_rows}, step[2] = {1, 1};
    return f(map, type, 2, const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
             CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct HeadIn {
    const void* x;
    const void* q;
};

template <typename T, typename O, int N>
sel_status launch(const HeadIn& in, const HeadArgs& args, cudaStream_t stream) {
    const int sms = device_sms();
    if (sms <= 0) return SEL_ECUDA;
    HeadArgs a = args;
    // every SM a run of whole weight copies, as even as 64 rows allow
    a.range = ceil_div(ceil_div(a.V, static_cast<uint64_t>(sms)), kBoxV) * kBoxV;
    CUtensorMap mw, mx;
    if (!make_map(&mw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, in.q, a.H / 2, a.V, kStageK / 2, kBoxV,
                  CU_TENSOR_MAP_SWIZZLE_64B) ||
        !make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, in.x, a.H, a.rows, kTileK, N, CU_TENSOR_MAP_SWIZZLE_128B))
        return SEL_ECUDA;
    if (!set_dynamic_smem(head_kernel<T, O, N>, Config<N>::kSmem)) return SEL_ECUDA;
    const cudaError_t e = launch_pdl(head_kernel<T, O, N>, dim3(ceil_div(a.V, a.range)), dim3(kNT), Config<N>::kSmem,
                                     stream, mw, mx, a);
    return e == cudaSuccess ? SEL_OK : SEL_ECUDA;
}

template <typename T, typename O>
sel_status launch_rows(const HeadIn& in, const HeadArgs& a, cudaStream_t stream) {
    if (a.rows <= 16) return launch<T, O, 16>(in, a, stream);
    if (a.rows <= 32) return launch<T, O, 32>(in, a, stream);
    return launch<T, O, 64>(in, a, stream);
}

template <typename T>
sel_status launch_out(int out_dtype, const HeadIn& in, const HeadArgs& a, cudaStream_t stream) {
    switch (out_dtype) {
        case SEL_F32: return launch_rows<T, float>(in, a, stream);
        case SEL_F16: return launch_rows<T, __half>(in, a, stream);
        default: return launch_rows<T, __nv_bfloat16>(in, a, stream);
    }
}

}  // namespace
}  // namespace sel

using namespace sel;

extern "C" sel_status sel_head_w4(const void* d_hidden, uint32_t rows, const uint8_t* d_q, const void* d_scales,
                                  const uint8_t* d_zeros, uint32_t group, int dtype, uint32_t V, uint32_t H,
                                  void* d_logits, int logits_dtype, uint64_t ld, cudaStream_t stream) {
    if (const sel_status s = check_w4(dtype, V, H, group); s != SEL_OK) return s;
    const uint32_t out_size = dtype_bytes(logits_dtype);
    if (out_size == 0 || ld < V || ld > SEL_MAX_LD) return SEL_EINVAL;
    if (rows == 0) return SEL_OK;
    if (!d_hidden || !d_q || !d_scales || !d_logits) return SEL_EINVAL;
    if (misaligned(d_hidden, 16) || misaligned(d_q, 16) || misaligned(d_scales, 2) || misaligned(d_logits, out_size))
        return SEL_EINVAL;
    if (rows > 0x7fffffffu) return SEL_EUNSUPPORTED;
    HeadArgs a{};
    a.scales = d_scales;
    a.zeros = d_zeros;
    a.out = d_logits;
    a.ld = ld;
    a.rows = rows;
    a.V = V;
    a.H = H;
    a.group = group;
    const HeadIn in{d_hidden, d_q};
    return dtype == SEL_F16 ? launch_out<__half>(logits_dtype, in, a, stream)
                            : launch_out<__nv_bfloat16>(logits_dtype, in, a, stream);
}
