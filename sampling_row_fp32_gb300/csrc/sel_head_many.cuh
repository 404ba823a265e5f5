// sel_head_many.cuh -- the 4-bit output head for more hidden rows than
// sel_head_few.cu takes; included once for each operand type.
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
//                 shared-memory stages of 256 columns (TMA, swizzled)
//   warps 4-19    unpack 128 columns of a row each: four 16-byte loads, nibbles
//                 to the type by placing them in the mantissa of 128 (bf16) or
//                 1024 (f16) and subtracting 128 + z (1024 + z), both exact;
//                 the tile goes to TMEM as the product's A operand
//   warp 3        brings the rows' scales and zero points
//   warps 1, 2    issue the products of a subtile each (A from TMEM, B =
//                 hidden states from shared memory, D in TMEM,
//                 double-buffered by group)
//   warps 20-27   read each group's D, add s * D to fp32 registers, and
//                 write the logits after the last group
// Every wait is bounded; one that runs out makes the CTA's logits NaN.
//
// What bounds it: not the copies (the matrix alone would take 77 us at 4,096 x
// 248,320) but instruction issue, 59 percent busy: 13 instructions a word of
// eight weights to unpack, a multiply-add for each D entry of a group, and the
// hand-overs between the roles. 4,096 x 248,320, groups of 64: 16 rows 117 us, 32
// rows 137, 49 rows 192-193 (3.0 TB/s, 520 TFLOP/s), 64 rows 195 (33 to 64 rows are
// one form, N = 64); 64 rows of 8,192 x 202,048, groups of 128: 253, with zero points
// 262-275. Folding the scales into the operand would take the epilogue out, and
// round every weight.
#pragma once

#include <type_traits>

#include "sel_head.cuh"
#include "sel_per_device.h"
#include "sel_tc.cuh"

namespace sel {
namespace {

constexpr uint32_t kSubV = 128;      // rows a subtile: TMEM lanes
constexpr uint32_t kAtomK = 64;      // columns of a 128-byte row of hidden states
constexpr uint32_t kABufs = kStageK / kUnitK;
constexpr uint32_t kACols = kUnitK / 2;  // TMEM columns of an A buffer
constexpr uint32_t kMaxStages = 10, kDBufs = 2;

// Warps: four of control, sixteen that unpack, eight of the epilogue; the
// registers of a launch (896 x 72) are split 56 / 56 / 112 between them.
constexpr int kUnpackWarp = 4, kEpilogueWarp = 20, kNT = 32 * 28;
constexpr int kLaunchRegs = 72, kControlRegs = 56, kUnpackRegs = 56, kEpilogueRegs = 112;
static_assert(4 * kControlRegs + 16 * kUnpackRegs + 8 * kEpilogueRegs <= 28 * kLaunchRegs);

// Zero points lie in their stage's slot. Scales have a ring of their own: the
// epilogue reads them well after the slot of their stage is free again.
constexpr uint32_t kZeroBytes = kTileV * EntryBytes<5>::kZeros;
constexpr uint32_t kScaleSlots = 5, kScaleBytes = kTileV * EntryBytes<5>::kScales;

template <int N>
struct Config {
    static constexpr uint32_t kXAtom = N * 128;  // 64 columns of N hidden rows
    static constexpr uint32_t kStageBytes = kWBytes + kStageK / kAtomK * kXAtom + kZeroBytes;
    static constexpr uint32_t kStages = 204 * 1024 / kStageBytes < kMaxStages ? 204 * 1024 / kStageBytes : kMaxStages;
    static constexpr uint32_t kSmem = 1024 + kStages * kStageBytes + kScaleSlots * kScaleBytes;
    static_assert(kSmem + 1024 <= 227 * 1024);
    // A D buffer's 64 columns hold up to 64 / N groups, handed over together.
    static constexpr uint32_t kBatch = 64 / N;
    static constexpr uint32_t kACol = 2 * kDBufs * 64;  // A buffers lie behind the D buffers
    static_assert(kACol + 2 * kABufs * kACols <= 512);
};

// ---------------------------------------------------------------------------
// tensor memory and tensor core primitives
// ---------------------------------------------------------------------------

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
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Eight nibbles to four pairs (columns 2 i, 2 i + 1) of q - z: byte i of the
// word and of the word shifted by a nibble into the pair's halves, the low
// nibble of each placed in the magic number, one subtraction.
template <typename T>
__device__ __forceinline__ void unpack8(uint32_t w, uint32_t zc, uint32_t* r) {
    const uint32_t u = w >> 4;
    // (in assembly: left to itself the compiler spends twice the instructions)
    asm("prmt.b32 %0, %1, %2, 0x4400;" : "=r"(r[0]) : "r"(w), "r"(u));
    asm("prmt.b32 %0, %1, %2, 0x5511;" : "=r"(r[1]) : "r"(w), "r"(u));
    asm("prmt.b32 %0, %1, %2, 0x6622;" : "=r"(r[2]) : "r"(w), "r"(u));
    asm("prmt.b32 %0, %1, %2, 0x7733;" : "=r"(r[3]) : "r"(w), "r"(u));
#pragma unroll
    for (uint32_t i = 0; i < 4; ++i) {
        asm("lop3.b32 %0, %0, 0x000F000F, %1, 0xEA;" : "+r"(r[i]) : "r"(Unpack<T>::kMagic));
        r[i] = Unpack<T>::sub(r[i], zc);
    }
}

template <int k>
using Log2 = std::integral_constant<int, k>;

struct Ctx {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t a_full[2][kABufs], a_empty[2][kABufs];
    uint64_t d_full[2][kDBufs], d_empty[2][kDBufs];
    uint64_t e_full[kScaleSlots], e_empty[kScaleSlots];
    uint64_t drain[2];
    uint32_t tmem;
    uint32_t err;
};

// Issues one subtile's products. The group is a template parameter so that a
// whole stage is straight-line code: this warp's instruction latencies, not
// the tensor cores, bound it otherwise.
template <typename T, int N>
struct MmaRole {
    using C = Config<N>;
    Ctx* c;
    unsigned char* ring;
    uint32_t s, a0, d0;
    bool leader;

    template <int kGroupLog2>
    __device__ __forceinline__ void run(uint32_t v_begin, uint32_t v_end, uint32_t blocks, uint32_t H) const {
        constexpr uint32_t kIdesc = (1u << 4) | (Unpack<T>::kType << 7) | (Unpack<T>::kType << 10) |
                                    (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(kSubV >> 4) << 24);
        constexpr uint32_t kPieces = (1u << kGroupLog2) / 32;  // pieces of 32 columns a group
        constexpr uint32_t kGroups = kUnitK >> kGroupLog2;     // groups a unit
        constexpr uint32_t kBatch = (C::kBatch < kGroups ? C::kBatch : kGroups) * kPieces;  // pieces a D buffer
        Ring<C::kStages> st;
        Ring<kDBufs> dr;
        uint32_t a_phase[kABufs] = {};
        for (uint32_t vt = v_begin; vt < v_end; vt += kTileV) {
            const bool active = s == 0 || v_end - vt > kSubV;
            for (uint32_t blk = 0; blk < blocks; ++blk) {
                for (uint32_t k = 0; k < H; k += kStageK) {
                    // a subtile without rows waits for the stage like its other
                    // readers, so that no arrival runs ahead into the slot's next use
                    wait(&c->full[st.i], st.phase, &c->err);
                    if (active) {
                        const uint64_t b = smem_desc(smem_u32(ring + st.i * C::kStageBytes + kWBytes));
                        const uint32_t left = H - k;
#pragma unroll
                        for (uint32_t u = 0; u < kABufs; ++u) {
                            if (u > 0 && u * kUnitK >= left) break;
                            wait(&c->a_full[s][u], a_phase[u], &c->err);
                            a_phase[u] ^= 1;
                            tc_fence_after();
#pragma unroll
                            for (uint32_t h = 0; h < kUnitK / 32; ++h) {
                                const uint32_t col = u * kUnitK + h * 32;
                                if (h > 0 && col >= left) break;  // whole groups only
                                if (h % kBatch == 0) {
                                    wait(&c->d_empty[s][dr.i], dr.phase ^ 1, &c->err);
                                    tc_fence_after();
                                }
                                // 32 columns: two products
                                const uint64_t bh = b + (col / kAtomK) * (C::kXAtom >> 4) + (col % kAtomK) / 8;
                                const uint32_t at = a0 + u * kACols + h * 16;
                                const uint32_t d = d0 + dr.i * 64 + h % kBatch / kPieces * N;
                                if (leader) {
                                    tc_mma(d, at, bh, kIdesc, h % kPieces != 0);
                                    tc_mma(d, at + 8, bh + 2, kIdesc, true);
                                }
                                if (h % kBatch == kBatch - 1 || col + 32 >= left) {
                                    if (leader) tc_commit(&c->d_full[s][dr.i]);
                                    dr.next();
                                }
                            }
                            if (leader) tc_commit(&c->a_empty[s][u]);
                        }
                        if (leader) tc_commit(&c->empty[st.i]);
                    } else if (leader) {
                        arrive(&c->empty[st.i]);
                    }
                    st.next();
                }
            }
        }
    }
};

// Brings the zero points of each stage into its slot and its scales into their
// ring. Loads go out before the waits for the slots.
template <int N>
struct EntryRole {
    using C = Config<N>;
    Ctx* c;
    unsigned char* ring;
    unsigned char* scales;

    template <int kGroupLog2, bool kZeros>
    __device__ __forceinline__ void run(const HeadArgs& a, uint32_t v_begin, uint32_t v_end, uint32_t blocks) const {
        using B = EntryBytes<kGroupLog2>;
        constexpr uint32_t kBatch = kGroupLog2 == 5 ? 4 : 8;  // rows a lane holds at a time
        const uint32_t lane = threadIdx.x & 31;
        const uint32_t groups = a.H >> kGroupLog2, stages = (a.H + kStageK - 1) / kStageK;
        const auto* s_base = static_cast<const unsigned char*>(a.scales);
        const uint32_t ws = entry_width(s_base, 2 * groups), wz = kZeros ? entry_width(a.zeros, groups) : 16;
        const bool wide = ws >= B::kScales && wz >= B::kZeros;
        Ring<C::kStages> st;
        Ring<kScaleSlots> er;
        for (uint32_t vt = v_begin; vt < v_end; vt += kTileV) {
            const uint32_t rows = min(kTileV, v_end - vt);
            const unsigned char* s_src = s_base + 2 * static_cast<uint64_t>(vt) * groups;
            const unsigned char* z_src = a.zeros + static_cast<uint64_t>(vt) * groups;
            for (uint32_t blk = 0; blk < blocks; ++blk) {
                for (uint32_t i = 0; i < stages; ++i) {
                    unsigned char* s_dst = scales + er.i * kScaleBytes;
                    unsigned char* z_dst = ring + (st.i + 1) * C::kStageBytes - kZeroBytes;
                    if (wide) {
#pragma unroll
                        for (uint32_t u = 0; u < kTileV / 32; u += kBatch) {
                            typename Word<B::kScales>::Type s[kBatch];
                            typename Word<B::kZeros>::Type z[kBatch];
                            const uint32_t u0 = u * 32 + lane;
                            if (kZeros) load_words<B::kZeros, B::kZeros, kBatch>(z, z_src, i * B::kZeros, groups, rows, u0);
                            load_words<B::kScales, B::kScales, kBatch>(s, s_src, i * B::kScales, 2 * groups, rows, u0);
                            if (u == 0) {
                                if (kZeros) wait(&c->empty[st.i], st.phase ^ 1, &c->err);
                                wait(&c->e_empty[er.i], er.phase ^ 1, &c->err);
                            }
                            if (kZeros) store_words<B::kZeros, B::kZeros, kBatch>(z_dst, z, rows, u0);
                            store_words<B::kScales, B::kScales, kBatch>(s_dst, s, rows, u0);
                        }
                    } else {
                        if (kZeros) wait(&c->empty[st.i], st.phase ^ 1, &c->err);
                        wait(&c->e_empty[er.i], er.phase ^ 1, &c->err);
                        if (kZeros) copy_rows<B::kZeros, 4>(z_dst, z_src, i * B::kZeros, groups, rows, wz);
                        copy_rows<B::kScales, 4>(s_dst, s_src, i * B::kScales, 2 * groups, rows, ws);
                    }
                    __syncwarp();
                    if (lane == 0) {
                        if (kZeros) arrive(&c->full[st.i]);
                        arrive(&c->e_full[er.i]);
                    }
                    st.next();
                    er.next();
                }
            }
        }
    }
};

// Unpacks one unit of every stage for 32 lanes of a subtile, into the A buffer
// of that unit.
template <typename T, int N>
struct UnpackRole {
    using C = Config<N>;
    Ctx* c;
    const unsigned char* ring;
    uint32_t s, unit, row, a0;  // row: within the tile

    template <bool kZeros, int kGroupLog2>
    __device__ __forceinline__ void run(uint32_t v_begin, uint32_t v_end, uint32_t blocks, uint32_t H) const {
        using B = EntryBytes<kGroupLog2>;
        const uint32_t lane = threadIdx.x & 31;
        // 16-byte chunk ch of a row lies at ch ^ (row & 7)
        const unsigned char* src = ring + row * (kStageK / 2);
        const uint32_t ch = unit * 4, sw = row & 7;
        const uint32_t ez = smem_u32(ring) + C::kStageBytes - kZeroBytes + row * B::kZeros;
        Ring<C::kStages> st;
        uint32_t phase = 0;  // of this unit's A buffer
        for (uint32_t vt = v_begin; vt < v_end; vt += kTileV) {
            const bool active = s == 0 || v_end - vt > kSubV;
            for (uint32_t blk = 0; blk < blocks; ++blk) {
                for (uint32_t k = 0; k < H; k += kStageK) {
                    wait(&c->full[st.i], st.phase, &c->err);
                    uint32_t zs = 0;  // the unit's zero points
                    if (kZeros) {
                        uint32_t v[(B::kZeros + 3) / 4];
                        read_entries<B::kZeros>(ez + st.i * C::kStageBytes, v);
                        if constexpr (kGroupLog2 == 5) zs = unit ? v[1] : v[0];
                        else zs = v[0] >> (unit * (B::kZeros / 2) * 8);
                    }
                    const bool mine = active && k + unit * kUnitK < H;  // the last stage may end before its second unit
                    if (mine) {
                        const unsigned char* p = src + st.i * C::kStageBytes;
                        uint4 q[4];
#pragma unroll
                        for (uint32_t j = 0; j < 4; ++j) q[j] = *reinterpret_cast<const uint4*>(p + (((ch + j) ^ sw) << 4));
#pragma unroll
                        for (uint32_t h = 0; h < 2; ++h) {
                            uint32_t r[32];
#pragma unroll
                            for (uint32_t j = 0; j < 2; ++j) {
                                const uint32_t z1 = kZeros ? (zs >> (8 * ((2 * h + j) * 32 >> kGroupLog2))) & 15 : 8;
                                const uint32_t zc = Unpack<T>::kMagic | z1 * 0x00010001u;
                                const uint4 v = q[2 * h + j];
                                unpack8<T>(v.x, zc, r + 16 * j);
                                unpack8<T>(v.y, zc, r + 16 * j + 4);
                                unpack8<T>(v.z, zc, r + 16 * j + 8);
                                unpack8<T>(v.w, zc, r + 16 * j + 12);
                            }
                            if (h == 0) {
                                wait(&c->a_empty[s][unit], phase ^ 1, &c->err);
                                tc_fence_after();
                            }
                            tmem_st32(a0 + h * 32, r);
                        }
                        tmem_wait_st();
                        tc_fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) {
                        if (mine) arrive(&c->a_full[s][unit]);
                        arrive(&c->empty[st.i]);
                    }
                    if (mine) phase ^= 1;
                    st.next();
                }
            }
        }
    }
};

// Adds one subtile's scaled group products for 32 matrix rows and writes them.
template <typename T, int N>
struct EpilogueRole {
    using C = Config<N>;
    Ctx* c;
    uint32_t scales;  // shared memory address of their ring
    void* out;
    int dtype;
    uint64_t ld;
    uint32_t rows, s, row, d0;

    template <int kGroupLog2>
    __device__ __forceinline__ void run(uint32_t v_begin, uint32_t v_end, uint32_t blocks, uint32_t H) const {
        using B = EntryBytes<kGroupLog2>;
        constexpr uint32_t kLd = N < 32 ? N : 32;  // columns of D a load
        constexpr uint32_t kPer = kUnitK >> kGroupLog2;
        constexpr uint32_t kBatch = C::kBatch < kPer ? C::kBatch : kPer;  // groups a D buffer
        const uint32_t lane = threadIdx.x & 31;
        const uint32_t es = scales + row * B::kScales;
        Ring<kDBufs> dr;
        Ring<kScaleSlots> er;
        for (uint32_t vt = v_begin; vt < v_end; vt += kTileV) {
            const bool active = s == 0 || v_end - vt > kSubV;
            for (uint32_t blk = 0; blk < blocks; ++blk) {
                float acc[N];
#pragma unroll
                for (int i = 0; i < N; ++i) acc[i] = 0.0f;
                for (uint32_t k = 0; k < H; k += kStageK) {
                    uint32_t sc[B::kScales / 4];
                    wait(&c->e_full[er.i], er.phase, &c->err);
                    read_entries<B::kScales>(es + er.i * kScaleBytes, sc);
                    __syncwarp();
                    if (lane == 0) arrive(&c->e_empty[er.i]);
                    er.next();
                    if (!active) continue;
#pragma unroll
                    for (uint32_t g0 = 0; g0 < B::kGroups; g0 += kBatch) {
                        if (g0 > 0 && k + (g0 << kGroupLog2) >= H) break;
                        wait(&c->d_full[s][dr.i], dr.phase, &c->err);
                        tc_fence_after();
#pragma unroll
                        for (uint32_t h = 0; h < kBatch * N / kLd; ++h) {
                            // columns h kLd .. of the buffer: of group g, from hidden row r
                            const uint32_t g = g0 + h * kLd / N, r = h * kLd % N;
                            const float sf = bits_f32<T>(entry16(sc, g));
                            uint32_t d[kLd];
                            tmem_ld(d0 + dr.i * 64 + h * kLd, d);
                            if (h == kBatch * N / kLd - 1) {  // the buffer is read
                                tc_fence_before();
                                __syncwarp();
                                if (lane == 0) arrive(&c->d_empty[s][dr.i]);
                            }
                            if (g == 0 || k + (g << kGroupLog2) < H) {  // (the last batch may be short)
#pragma unroll
                                for (uint32_t i = 0; i < kLd; ++i) acc[r + i] = fmaf(sf, __uint_as_float(d[i]), acc[r + i]);
                            }
                        }
                        dr.next();
                    }
                }
                if (active && vt + row < v_end) {
                    const uint32_t n = rows - blk * N;
                    auto write = [&](auto* o) {
                        o += static_cast<uint64_t>(blk) * N * ld + vt + row;
#pragma unroll
                        for (uint32_t i = 0; i < N; ++i)
                            if (i < n) o[i * ld] = from_f32<std::remove_pointer_t<decltype(o)>>(acc[i]);
                    };
                    if (dtype == SEL_F32) write(static_cast<float*>(out));
                    else if (dtype == SEL_F16) write(static_cast<__half*>(out));
                    else write(static_cast<__nv_bfloat16*>(out));
                }
            }
        }
    }
};

template <typename T, int N>
__global__ void __launch_bounds__(kNT, 1)
    head_kernel(const __grid_constant__ CUtensorMap map_tile, const __grid_constant__ CUtensorMap map_box,
                const __grid_constant__ CUtensorMap map_x, HeadArgs a) {
    using C = Config<N>;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char* scales = ring + C::kStages * C::kStageBytes;
    __shared__ Ctx c;
    // (broadcasts: the compiler then keeps what follows from them in uniform registers)
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);

    if (tid == 0) {
        for (uint32_t i = 0; i < C::kStages; ++i) {
            mbar_init(&c.full[i], a.zeros ? 2 : 1);  // the copies, and the helper's zero points
            mbar_init(&c.empty[i], 16 + 2);  // the unpacking warps and the products
        }
        for (uint32_t s = 0; s < 2; ++s) {
            mbar_init(&c.drain[s], 1);
            for (uint32_t i = 0; i < kABufs; ++i) {
                mbar_init(&c.a_full[s][i], 4);
                mbar_init(&c.a_empty[s][i], 1);
            }
            for (uint32_t i = 0; i < kDBufs; ++i) {
                mbar_init(&c.d_full[s][i], 1);
                mbar_init(&c.d_empty[s][i], 4);
            }
        }
        for (uint32_t i = 0; i < kScaleSlots; ++i) {
            mbar_init(&c.e_full[i], 1);
            mbar_init(&c.e_empty[i], 8);
        }
        c.err = 0;
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&c.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    const uint32_t v_begin = blockIdx.x * a.range, v_end = min(a.V, v_begin + a.range);
    if (warp == 0 && elect_one() && v_end - v_begin >= kTileV) {  // the first stages, while the launch before ends
        const uint32_t n = min(C::kStages, (a.H + kStageK - 1) / kStageK);
        for (uint32_t i = 0; i < n; ++i) tma_prefetch_2d(&map_tile, i * (kStageK / 2), v_begin);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(kFull, c.tmem, 0);
    pdl_wait();
    pdl_trigger();
    const uint32_t blocks = (a.rows + N - 1) / N;  // blocks of hidden rows
    const uint32_t quarter = warp & 3;

    if (warp < kUnpackWarp) {
        regs_dec<kControlRegs>();
        // The control warps stay together, so that addresses and descriptors live
        // in uniform registers; one elected lane issues. (Issued by a lane on its
        // own, a stage's copies took 1.3k clocks, its products 1.7k, against the
        // 750 that the weights' bytes take at the copy rate.)
        const bool leader = elect_one();
        if (warp == 0) {
            const uint32_t stages = (a.H + kStageK - 1) / kStageK;
            Ring<C::kStages> st;
            uint32_t issued = 0;
            bool ok = true;
            for (uint32_t vt = v_begin; vt < v_end && ok; vt += kTileV) {
                const uint32_t boxes = (min(kTileV, v_end - vt) + kBoxV - 1) / kBoxV;
                for (uint32_t blk = 0; blk < blocks && ok; ++blk) {
                    for (uint32_t i = 0; i < stages; ++i) {
                        ok = __all_sync(kFull, mbar_wait(&c.empty[st.i], st.phase ^ 1));
                        if (!ok) break;
                        unsigned char* dst = ring + st.i * C::kStageBytes;
                        uint64_t* full = &c.full[st.i];
                        const uint32_t atoms = min(kStageK / kAtomK, (a.H - i * kStageK + kAtomK - 1) / kAtomK);
                        if (leader) {
                            expect_tx(full, boxes * kBoxV * (kStageK / 2) + atoms * C::kXAtom);
                            if (boxes == kTileV / kBoxV) {
                                tma_2d(dst, &map_tile, i * (kStageK / 2), vt, full);
                            } else {
                                for (uint32_t b = 0; b < boxes; ++b)
                                    tma_2d(dst + b * kBoxV * (kStageK / 2), &map_box, i * (kStageK / 2), vt + b * kBoxV,
                                           full);
                            }
                            for (uint32_t at = 0; at < atoms; ++at)
                                tma_2d(dst + kWBytes + at * C::kXAtom, &map_x, i * kStageK + at * kAtomK, blk * N, full);
                        }
                        ++issued;
                        st.next();
                    }
                }
            }
            // every copy has landed before the CTA may end
            if (leader) {
                for (uint32_t i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
                    if (!mbar_wait(&c.full[i % C::kStages], (i / C::kStages) & 1)) ok = false;
                if (!ok) c.err = 1;
            }
        } else if (warp == 1 || warp == 2) {
            const uint32_t s = warp - 1;
            const MmaRole<T, N> role{&c, ring, s, tmem + C::kACol + s * kABufs * kACols, tmem + s * kDBufs * 64, leader};
            if (a.group_log2 == 7) role.template run<7>(v_begin, v_end, blocks, a.H);
            else if (a.group_log2 == 6) role.template run<6>(v_begin, v_end, blocks, a.H);
            else role.template run<5>(v_begin, v_end, blocks, a.H);
            // no product is in flight when the tensor memory is given back
            if (leader) tc_commit(&c.drain[s]);
            if (!mbar_wait(&c.drain[s], 0)) c.err = 1;
        } else {
            const EntryRole<N> role{&c, ring, scales};
            auto copy = [&](auto log2, auto zeros) {
                role.template run<decltype(log2)::value, decltype(zeros)::value>(a, v_begin, v_end, blocks);
            };
            using Yes = std::true_type;
            using No = std::false_type;
            if (a.group_log2 == 7) a.zeros ? copy(Log2<7>{}, Yes{}) : copy(Log2<7>{}, No{});
            else if (a.group_log2 == 6) a.zeros ? copy(Log2<6>{}, Yes{}) : copy(Log2<6>{}, No{});
            else a.zeros ? copy(Log2<5>{}, Yes{}) : copy(Log2<5>{}, No{});
        }
        __syncwarp();
    } else if (warp < kEpilogueWarp) {
        regs_dec<kUnpackRegs>();
        const uint32_t wg = (warp - kUnpackWarp) / 4, s = wg & 1, unit = wg >> 1;
        const UnpackRole<T, N> role{&c, ring, s, unit, s * kSubV + quarter * 32 + lane,
                                    tmem + (quarter << 21) + C::kACol + (s * kABufs + unit) * kACols};
        if (!a.zeros) role.template run<false, 7>(v_begin, v_end, blocks, a.H);
        else if (a.group_log2 == 7) role.template run<true, 7>(v_begin, v_end, blocks, a.H);
        else if (a.group_log2 == 6) role.template run<true, 6>(v_begin, v_end, blocks, a.H);
        else role.template run<true, 5>(v_begin, v_end, blocks, a.H);
    } else {
        regs_inc<kEpilogueRegs>();
        const uint32_t s = (warp - kEpilogueWarp) / 4;
        const EpilogueRole<T, N> role{&c, smem_u32(scales), a.out, a.out_dtype, a.ld, a.rows, s,
                                         s * kSubV + quarter * 32 + lane, tmem + (quarter << 21) + s * kDBufs * 64};
        if (a.group_log2 == 7) role.template run<7>(v_begin, v_end, blocks, a.H);
        else if (a.group_log2 == 6) role.template run<6>(v_begin, v_end, blocks, a.H);
        else role.template run<5>(v_begin, v_end, blocks, a.H);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    if (c.err) {  // a wait ran out: nothing this CTA wrote can be trusted
        for (uint32_t r = 0; r < a.rows; ++r)
            for (uint32_t v = v_begin + tid; v < v_end; v += kNT)
                store_as(a.out, a.out_dtype, r * a.ld + v, __uint_as_float(0x7FC00000u));
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

template <typename T, int N>
sel_status launch(const HeadIn& in, const HeadArgs& args, cudaStream_t stream) {
    const int sms = device_sms();
    if (sms <= 0) return SEL_ECUDA;
    HeadArgs a = args;
    a.range = head_range(a.V, sms);
    CUtensorMap mt, mb, mx;
    if (!make_weight_map(&mt, in.q, a.V, a.H, kTileV) || !make_weight_map(&mb, in.q, a.V, a.H, kBoxV) ||
        !make_map(&mx, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, in.x, a.H, a.rows, kAtomK, N, CU_TENSOR_MAP_SWIZZLE_128B))
        return SEL_ECUDA;
    // the split of the registers counts on what the launch has
    static PerDevice<int> registers;
    int dev = -1, regs = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || !registers.get(dev, regs, [](int& n) {
            cudaFuncAttributes f{};
            if (cudaFuncGetAttributes(&f, head_kernel<T, N>) != cudaSuccess) return false;
            n = f.numRegs;
            return true;
        }))
        return SEL_ECUDA;
    if (regs != kLaunchRegs || !dynamic_smem_once<head_kernel<T, N>>(Config<N>::kSmem)) return SEL_ECUDA;
    const cudaError_t e = launch_pdl(head_kernel<T, N>, dim3(ceil_div(a.V, a.range)), dim3(kNT), Config<N>::kSmem,
                                     stream, mt, mb, mx, a);
    return e == cudaSuccess ? SEL_OK : SEL_ECUDA;
}

}  // namespace

template <typename T>
sel_status head_many(const HeadIn& in, const HeadArgs& a, cudaStream_t stream) {
    if (a.rows <= 16) return launch<T, 16>(in, a, stream);
    if (a.rows <= 32) return launch<T, 32>(in, a, stream);
    return launch<T, 64>(in, a, stream);
}

}  // namespace sel
