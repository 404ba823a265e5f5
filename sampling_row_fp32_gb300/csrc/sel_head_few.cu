// sel_head_few.cu -- the 4-bit output head for at most 8 hidden rows (plain
// decoding, a few sequences), where the weights' bytes are the whole cost.
//
// The same sums as sel_head_many.cuh, with the products on warp-level matrix
// instructions whose A operand (the weights) comes from registers: an
// unpacked word needs no trip through tensor memory, and because this kernel
// lays out the hidden rows, a pair of operand columns may be any two columns.
// Nibbles i and i + 4 of a word are 16 bits apart, so a mask leaves them as a
// pair. What bounds the kernel then is the integer pipe, at half an
// instruction a clock: 9 instructions a word for neighbouring columns, 7 for
// these pairs, and 5 with f16 operands, where the ten bits of the mantissa
// also hold a nibble four bits higher up (times 1/16, exact), so that only one
// shift is left. bf16 hidden rows therefore become f16 where that loses
// nothing: a row is scaled by the power of two that brings its largest value
// under 2^15, and bf16's eight significant bits fit f16 down to 2^-17, a span
// of 2^32. A row with nonzero values below that keeps the whole call on bf16
// operands.
//
// The hidden rows sit in shared memory for the CTA's whole life, in the order
// (0,4)(1,5)(2,6)(3,7) of each eight columns. A CTA per SM walks its run of
// matrix rows in tiles of equal height (up to 352) through a ring of stages of
// 256 columns that one warp fills (TMA); warp w of the others owns rows 16 w ..
// 16 w + 15 of a tile over all columns, so nothing is exchanged between warps.
// One row of 4,096 x 248,320 takes 93 us with groups of 128 and 99 with 64, 5.6
// and 5.4 TB/s; the matrix's bytes alone would take 77 and 80.
#include <type_traits>

#include "sel_head.cuh"

namespace sel {
namespace {

constexpr uint32_t kMaxTile = 352;                    // 22 warps
constexpr uint32_t kHelpers = 4;                      // warps that bring the group entries
constexpr int kMaxNT = 32 * (kMaxTile / 16 + 1 + kHelpers);  // and the copying warp
constexpr uint32_t kRowBytes = kStageK / 2;
constexpr uint32_t kMaxStages = 8, kMinStages = 3;
constexpr uint32_t kSmemBytes = 225 * 1024;  // alignment, ring and hidden rows

struct Ctx {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint32_t largest[8];  // of a hidden row: the magnitude's bits
    uint32_t err;
};

template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma<__nv_bfloat16>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma<__half>(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The constants that take nibbles out of their magic numbers: 128 + z for bf16;
// for f16 1024 + z, and 64 + z for a nibble four bits up, after the factor 1/16.
template <typename E>
struct ZeroPoint {
    uint32_t low, high;
    __device__ __forceinline__ explicit ZeroPoint(uint32_t z) {
        const uint32_t zz = z * 0x00010001u;
        low = Unpack<E>::kMagic | zz;
        high = 0xD400D400u | (zz << 4);  // -(64 + z)
    }
};

// Nibbles i and i + 4 of a word, less the zero point, as the pair r[i].
template <typename E>
__device__ __forceinline__ void unpack_pairs(uint32_t w, const ZeroPoint<E>& z, uint32_t (&r)[4]) {
    if constexpr (Unpack<E>::kType == 0) {
        const uint32_t u = w >> 8;
        asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(r[0]) : "r"(w), "r"(Unpack<E>::kMagic));
        asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0xEA;" : "=r"(r[1]) : "r"(w), "r"(Unpack<E>::kMagic));
        asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(r[2]) : "r"(u), "r"(Unpack<E>::kMagic));
        asm("lop3.b32 %0, %1, 0x00F000F0, %2, 0xEA;" : "=r"(r[3]) : "r"(u), "r"(Unpack<E>::kMagic));
        r[0] = Unpack<E>::sub(r[0], z.low);
        r[2] = Unpack<E>::sub(r[2], z.low);
        asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(r[1]) : "r"(0x2C002C00u), "r"(z.high));  // 1/16
        asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(r[3]) : "r"(0x2C002C00u), "r"(z.high));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(r[i]) : "r"(w >> (4 * i)), "r"(Unpack<E>::kMagic));
            r[i] = Unpack<E>::sub(r[i], z.low);
        }
    }
}

struct FewArgs {
    HeadArgs a;
    uint32_t tile;    // rows a tile, a multiple of 16
    uint32_t stages;  // slots of the ring
};

// Power of two that brings a row of bf16 values, the largest of magnitude bits
// `m`, under 2^15 (exponent clamped so that it and its inverse are normal).
__device__ __forceinline__ int row_shift(uint32_t m) {
    const int e = static_cast<int>(m >> 7) - 127;  // 2^e <= largest < 2^(e + 1)
    return m ? min(max(14 - e, -120), 120) : 0;
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

__device__ __forceinline__ void mul2(float& a, float& b, const float (&f)[2]) {
    asm("{\n\t.reg .b64 x, y;\n\t"
        "mov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\t"
        "mul.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(f[0]), "f"(f[1]));
}

// The consuming warps: operands of type E (T, or f16 for a bf16 T).
template <typename T, typename E, int kGroupLog2, bool kZeros>
__device__ __forceinline__ void consume(Ctx& c, uint32_t ring, uint32_t entries, uint32_t xs, const FewArgs& f, uint32_t v_begin,
                                        uint32_t v_end) {
    using B = EntryBytes<kGroupLog2>;
    constexpr uint32_t kBlocks = (1u << kGroupLog2) / 32;  // blocks of 32 columns a group
    const HeadArgs& a = f.a;
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
    const uint32_t g = lane >> 2, t = lane & 3;
    const uint32_t row = warp * 16 + g;  // and row + 8
    const uint32_t stages = (a.H + kStageK - 1) / kStageK;
    // chunk ch of a row lies at ch ^ (row & 7); rows r and r + 8 agree in that
    const uint32_t w0 = ring + row * kRowBytes + t * 4 + (g << 4);
    // operand columns past the last hidden row repeat it; nothing reads their sums
    const uint32_t x0 = xs + min(g, a.rows - 1) * 64 + t * 16;
    const uint32_t entry_bytes = f.tile * (B::kScales + (kZeros ? B::kZeros : 0));  // a slot's
    const uint32_t e0 = entries + row * B::kScales, ez = entries + f.tile * B::kScales + row * B::kZeros;
    const uint32_t x_block = a.rows * 64, slot_bytes = f.tile * kRowBytes;
    // Sums go back to scale before the group's scale meets them, as far as they
    // stay in range: a group's is below 2^26, so by up to 2^100. What is left, for
    // rows that were scaled down by more, follows at the end. Nothing in between
    // overflows that unscaled sums would not, and nothing gets lost below fp32's
    // smallest normal (a group's least nonzero sum is 2^-24, and it back by 2^100
    // meets scales of 2^-133 at the least).
    constexpr bool kScaled = !std::is_same_v<T, E>;
    float before[2], after[2];
    if constexpr (kScaled) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int sh = row_shift(c.largest[min(2 * t + e, a.rows - 1)]);
            before[e] = exp2i(min(-sh, 100));
            after[e] = exp2i(max(-sh - 100, 0));
        }
    }
    uint32_t slot = 0, phase = 0;
    for (uint32_t vt = v_begin; vt < v_end; vt += f.tile) {
        const bool active = warp * 16 < v_end - vt;
        float acc[4] = {};
        for (uint32_t i = 0; i < stages; ++i) {
            wait(&c.full[slot], phase, &c.err);
            if (active) {
                const uint32_t wp = w0 + slot * slot_bytes;
                const uint32_t xp = i * (kStageK / 32) * x_block;
                uint32_t sc[2][B::kScales / 4], zp[2][(B::kZeros + 3) / 4];
#pragma unroll
                for (uint32_t h = 0; h < 2; ++h) {
                    read_entries<B::kScales>(e0 + slot * entry_bytes + 8 * h * B::kScales, sc[h]);
                    if (kZeros) read_entries<B::kZeros>(ez + slot * entry_bytes + 8 * h * B::kZeros, zp[h]);
                }
                float d[4];
#pragma unroll
                for (uint32_t b = 0; b < kStageK / 32; ++b) {
                    const uint32_t grp = b / kBlocks;
                    uint32_t wa, wb;
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(wa) : "r"(wp ^ (b << 4)));
                    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(wb) : "r"((wp ^ (b << 4)) + 8 * kRowBytes));
                    const ZeroPoint<E> za(kZeros ? zero_point(zp[0], grp) : 8), zb(kZeros ? zero_point(zp[1], grp) : 8);
                    uint32_t pa[4], pb[4];
                    unpack_pairs<E>(wa, za, pa);
                    unpack_pairs<E>(wb, zb, pb);
                    const uint32_t a01[4] = {pa[0], pb[0], pa[1], pb[1]}, a23[4] = {pa[2], pb[2], pa[3], pb[3]};
                    uint32_t xv[4];
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(xv[0]), "=r"(xv[1]), "=r"(xv[2]), "=r"(xv[3])
                                 : "r"(x0 + xp + b * x_block));
                    if (b % kBlocks == 0) d[0] = d[1] = d[2] = d[3] = 0.0f;
                    mma<E>(d, a01, xv[0], xv[1]);
                    mma<E>(d, a23, xv[2], xv[3]);
                    if (b % kBlocks == kBlocks - 1) {
                        const float sa = bits_f32<T>(entry16(sc[0], grp)), sb = bits_f32<T>(entry16(sc[1], grp));
                        if constexpr (kScaled) {
                            mul2(d[0], d[1], before);
                            mul2(d[2], d[3], before);
                        }
                        acc[0] = fmaf(sa, d[0], acc[0]);
                        acc[1] = fmaf(sa, d[1], acc[1]);
                        acc[2] = fmaf(sb, d[2], acc[2]);
                        acc[3] = fmaf(sb, d[3], acc[3]);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) arrive(&c.empty[slot]);
            if (++slot == f.stages) {
                slot = 0;
                phase ^= 1;
            }
        }
        // D's element (row g or g + 8, hidden row 2 t or 2 t + 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t r = 2 * t + (e & 1), v = vt + row + 8 * (e >> 1);
            if constexpr (kScaled) acc[e] *= after[e & 1];
            if (active && r < a.rows && v < v_end) store_as(a.out, a.out_dtype, r * a.ld + v, acc[e]);
        }
    }
}

template <typename T, int kGroupLog2, bool kZeros>
__global__ void __launch_bounds__(kMaxNT, 1)
    head_few_kernel(const __grid_constant__ CUtensorMap map, const T* x, const __grid_constant__ FewArgs f) {
    const HeadArgs& a = f.a;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* ring = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t slot_bytes = f.tile * kRowBytes;
    unsigned char* entries = ring + f.stages * slot_bytes;
    const uint32_t entry_bytes = f.tile * (EntryBytes<kGroupLog2>::kScales + (kZeros ? EntryBytes<kGroupLog2>::kZeros : 0));
    unsigned char* xs = entries + f.stages * entry_bytes;
    __shared__ Ctx c;
    const uint32_t tid = threadIdx.x, warp = __shfl_sync(kFull, tid >> 5, 0);
    const uint32_t workers = f.tile / 16;  // consuming warps; the next ones copy
    if (tid == 0) {
        for (uint32_t i = 0; i < f.stages; ++i) {
            mbar_init(&c.full[i], 1 + 1);  // the weights' copy and a helper
            mbar_init(&c.empty[i], workers);
        }
        c.err = 0;
    }
    if (tid < 8) c.largest[tid] = 0;
    const uint32_t v_begin = blockIdx.x * a.range, v_end = min(a.V, v_begin + a.range);
    if (warp == workers && elect_one()) {  // the first stages, while the launch before ends
        const uint32_t n = min(f.stages, (a.H + kStageK - 1) / kStageK);
        for (uint32_t i = 0; i < n; ++i) {
            tma_prefetch_2d(&map, i * kRowBytes, v_begin);
            if (v_begin + f.tile / 2 < v_end) tma_prefetch_2d(&map, i * kRowBytes, v_begin + f.tile / 2);
        }
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    if (warp == workers) {
        const uint32_t stages = (a.H + kStageK - 1) / kStageK;
        const bool leader = elect_one();
        uint32_t issued = 0, slot = 0, phase = 0;
        bool ok = true;
        for (uint32_t vt = v_begin; vt < v_end && ok; vt += f.tile) {
            for (uint32_t i = 0; i < stages; ++i) {
                ok = __all_sync(kFull, mbar_wait(&c.empty[slot], phase ^ 1));
                if (!ok) break;
                if (leader) {
                    unsigned char* dst = ring + slot * slot_bytes;
                    expect_tx(&c.full[slot], slot_bytes);
                    tma_2d(dst, &map, i * kRowBytes, vt, &c.full[slot]);
                    tma_2d(dst + slot_bytes / 2, &map, i * kRowBytes, vt + f.tile / 2, &c.full[slot]);
                }
                ++issued;
                if (++slot == f.stages) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        // every copy has landed before the CTA may end
        if (leader) {
            for (uint32_t i = issued > f.stages ? issued - f.stages : 0; i < issued; ++i)
                if (!mbar_wait(&c.full[i % f.stages], (i / f.stages) & 1)) ok = false;
            if (!ok) c.err = 1;
        }
        __syncwarp();
    } else if (warp > workers) {
        // No more helpers take turns than the ring has slots: one that ran a whole
        // round ahead would take a slot's phase before last for its last.
        const uint32_t lane = tid & 31, helper = warp - workers - 1, helpers = min(kHelpers, f.stages);
        if (helper < helpers) copy_entries<kGroupLog2, kZeros, kMaxTile / 32>(
            a, entries, entry_bytes, f.tile, f.stages, helper, helpers, v_begin, v_end,
            [&](uint32_t slot, uint32_t phase) { wait(&c.empty[slot], phase ^ 1, &c.err); },
            [&](uint32_t slot) {
                if (lane == 0) arrive(&c.full[slot]);
            });
    } else {
        // Block kb of 32 columns, row n, 16 bytes for each of the four lanes that
        // share a row of an operand; zeros past the last column.
        const uint32_t nt = 32 * workers;
        const uint32_t vecs = (a.H + kStageK - 1) / kStageK * (kStageK / 8) * a.rows;
        auto bar = [&] { asm volatile("bar.sync 1, %0;" ::"r"(nt) : "memory"); };
        auto load = [&](uint32_t i, uint32_t& n) {
            const uint32_t b = (i >> 2) / a.rows, k = b * 32 + (i & 3) * 8;
            n = (i >> 2) - b * a.rows;
            return k < a.H ? *reinterpret_cast<const uint4*>(x + static_cast<uint64_t>(n) * a.H + k) : make_uint4(0, 0, 0, 0);
        };
        auto store = [&](uint32_t i, const uint4& u) {
            reinterpret_cast<uint4*>(xs)[i] = make_uint4(__byte_perm(u.x, u.z, 0x5410), __byte_perm(u.x, u.z, 0x7632),
                                                         __byte_perm(u.y, u.w, 0x5410), __byte_perm(u.y, u.w, 0x7632));
        };
        bool as_f16 = false;
        if constexpr (std::is_same_v<T, __nv_bfloat16>) {
            // each row's largest finite magnitude, then the row as f16 where that
            // is exact
            for (uint32_t i = tid; i < vecs; i += nt) {
                uint32_t n, m = 0;
                const uint4 u = load(i, n);
                const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t lo = w[j] & 0x7FFFu, hi = (w[j] >> 16) & 0x7FFFu;
                    if (lo < 0x7F80u) m = max(m, lo);
                    if (hi < 0x7F80u) m = max(m, hi);
                }
                if (m > *const_cast<volatile uint32_t*>(&c.largest[n])) atomicMax(&c.largest[n], m);
            }
            bar();
            bool exact = true;
            for (uint32_t i = tid; i < vecs; i += nt) {
                uint32_t n;
                uint4 u = load(i, n);
                const int sh = row_shift(c.largest[n]);
                const float up = exp2i(sh);
                uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float lo = __uint_as_float(w[j] << 16), hi = __uint_as_float(w[j] & 0xFFFF0000u);
                    const __half2 y = __floats2half2_rn(lo * up, hi * up);
                    const float2 back = __half22float2(y);
                    exact = exact && (back.x == lo * up || lo != lo) && (back.y == hi * up || hi != hi) &&
                            (lo == 0.0f) == (back.x == 0.0f) && (hi == 0.0f) == (back.y == 0.0f);
                    w[j] = *reinterpret_cast<const uint32_t*>(&y);
                }
                store(i, make_uint4(w[0], w[1], w[2], w[3]));
            }
            int any;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\t"
                "setp.ne.s32 p, %1, 0;\n\t"
                "bar.red.and.pred q, 1, %2, p;\n\t"
                "selp.s32 %0, 1, 0, q;\n\t}"
                : "=r"(any)
                : "r"(static_cast<int>(exact)), "r"(nt)
                : "memory");
            as_f16 = any != 0;
        }
        if (!as_f16) {
            for (uint32_t i = tid; i < vecs; i += nt) {
                uint32_t n;
                const uint4 u = load(i, n);
                store(i, u);
            }
            bar();
        }
        const uint32_t rs = smem_u32(ring), es = smem_u32(entries), xa = smem_u32(xs);
        if constexpr (std::is_same_v<T, __nv_bfloat16>) {
            if (as_f16) consume<T, __half, kGroupLog2, kZeros>(c, rs, es, xa, f, v_begin, v_end);
            else consume<T, T, kGroupLog2, kZeros>(c, rs, es, xa, f, v_begin, v_end);
        } else {
            consume<T, T, kGroupLog2, kZeros>(c, rs, es, xa, f, v_begin, v_end);
        }
    }
    __syncthreads();
    if (c.err) {  // a wait ran out: nothing this CTA wrote can be trusted
        for (uint32_t r = 0; r < a.rows; ++r)
            for (uint32_t v = v_begin + tid; v < v_end; v += blockDim.x)
                store_as(a.out, a.out_dtype, r * a.ld + v, __uint_as_float(0x7FC00000u));
    }
}

template <typename T, int kGroupLog2, bool kZeros>
sel_status launch(const HeadIn& in, const HeadArgs& args, cudaStream_t stream) {
    const int sms = device_sms();
    if (sms <= 0) return SEL_ECUDA;
    FewArgs f{args, 0, 0};
    const uint32_t x_bytes = args.rows * ceil_div(args.H, kStageK) * kStageK * 2;
    const uint32_t ring_bytes = kSmemBytes - 1024 - x_bytes;
    // the SMs' even share of the rows in tiles of one height, as high as
    // kMinStages slots allow
    const uint32_t row_bytes = kRowBytes + entry_row_bytes(kGroupLog2, kZeros);
    const uint32_t most = ring_bytes / kMinStages / row_bytes / 16 * 16;
    const uint32_t share = ceil_div(args.V, static_cast<uint64_t>(sms)), tiles = ceil_div(share, most < kMaxTile ? most : kMaxTile);
    f.tile = ceil_div(ceil_div(share, tiles), 16) * 16;
    f.a.range = tiles * f.tile;
    f.stages = ring_bytes / (f.tile * row_bytes);
    if (f.stages > kMaxStages) f.stages = kMaxStages;
    CUtensorMap map;
    if (!make_weight_map(&map, in.q, args.V, args.H, f.tile / 2)) return SEL_ECUDA;
    constexpr auto kernel = head_few_kernel<T, kGroupLog2, kZeros>;
    if (!dynamic_smem_once<kernel>(kSmemBytes)) return SEL_ECUDA;
    const cudaError_t e = launch_pdl(kernel, dim3(ceil_div(args.V, f.a.range)), dim3(32 * (f.tile / 16 + 1 + kHelpers)),
                                     1024 + f.stages * f.tile * row_bytes + x_bytes, stream, map,
                                     static_cast<const T*>(in.x), f);
    return e == cudaSuccess ? SEL_OK : SEL_ECUDA;
}

template <typename T, bool kZeros>
sel_status launch_group(const HeadIn& in, const HeadArgs& a, cudaStream_t stream) {
    if (a.group_log2 == 7) return launch<T, 7, kZeros>(in, a, stream);
    if (a.group_log2 == 6) return launch<T, 6, kZeros>(in, a, stream);
    return launch<T, 5, kZeros>(in, a, stream);
}

template <typename T>
sel_status launch_zeros(const HeadIn& in, const HeadArgs& a, cudaStream_t stream) {
    return a.zeros ? launch_group<T, true>(in, a, stream) : launch_group<T, false>(in, a, stream);
}

}  // namespace

sel_status head_few(int dtype, const HeadIn& in, const HeadArgs& a, cudaStream_t stream) {
    return dtype == SEL_F16 ? launch_zeros<__half>(in, a, stream) : launch_zeros<__nv_bfloat16>(in, a, stream);
}

}  // namespace sel
