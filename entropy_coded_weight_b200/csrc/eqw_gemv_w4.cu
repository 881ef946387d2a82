// Matrix-vector products with 4-bit weights and group scales: eq_gemv_w4.
//
//   y[t, r] = sum_g s[r, g] * sum_{c in group g} w(q[r, c]) * x[t, c],  t < tokens <= 32
//   w(q) = q - 8, q - zero[r, g] (0 to 127), or table[q] (16 bf16 values)
// Every w is exact in bf16, so a group's inner sum runs on the tensor cores
// (tcgen05.mma kind::f16, exact products, fp32 accumulator) and its scale
// multiplies it once, in fp32, when the sum leaves tensor memory.
//
// Bound by memory (half a byte per weight, read once) as long as decoding keeps
// up: at 6.5 TB/s an SM gets 46 weights per clock and has 4 issue slots for
// them, so an fp32 multiply-add per weight and token is out of reach, and so is
// mma.sync, whose every instruction takes eight issue slots here.  With the
// products on tcgen05 the threads only decode: 11 instructions per 8 codes.
//
// One CTA per SM, a tile of up to 128 rows (a thread per row: tensor-memory
// lane = row), K in slabs of 256 or 128 columns.  Roles:
//   loader    one lane: the codes of a slab (rows x 128 or 64 bytes, swizzled)
//             by TMA into a deep ring ("landed" / "read")
//   decoders  PARTS groups of four warps, group p taking slabs p, p + PARTS, ...:
//             a thread decodes its row's codes to bf16 and stores them to
//             tensor memory (A of the product, one stage per group), then
//             "ready".  Before its next slab it takes the finished sums of
//             the last one ("done") and adds scale x sum to its fp32 totals.
//   products  PARTS warps, one per stage: the slab of x as B (K-major,
//             128-byte swizzle) in shared memory, the 8 columns of a code word
//             in the order in which the codes pair up in a register (i and
//             i + 4, or i and i + 1 through the table); then, after "ready", the
//             products (K = 16) into one accumulator per group of columns and a
//             commit to "done".  (One warp issuing for all stages took 500
//             clocks per slab, more than memory.)
// A group's stage (A, B and accumulators) is reused by the same group only, so
// "done" is the only barrier behind the product.  The groups' totals meet in
// shared memory in a fixed order; where there are fewer row tiles than SMs, the
// CTAs of a cluster share K and their totals meet over distributed shared memory.
//
// Measured (B200): one token x 18944 x 8192, groups of 128: 20 us, 4.0 TB/s; 75776 x
// 8192: 67 to 75 us for one token, 75 for eight, 84 for 16 (memory: 49).  The decoders
// bound it: issue slots, logic pipe and tensor pipe are 55, 58 and 13 % busy, the rest
// are their waits.  The same product with mma.sync took 81 us for one token and 97
// for eight.
// Those rows fill the SMs evenly (one and four tiles of 128 each).  28672 x 8192 is 224
// tiles, two rounds for 1.5 rounds' rows: eight tokens with zero points 37 to 39 us
// (memory: 19), 32 tokens 67.  Groups of 32, whose sums leave tensor memory four times as
// often: 49 us for one token, 60 for eight, 93 for 32 with a table.  4096 x 4096 takes
// 6.3 us (memory: 1.3), most of it start and end.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cstring>
#include <vector>

#include "eqw_device.cuh"
#include "eqw_launch.cuh"
#include "eqw_tc.cuh"

namespace {

constexpr uint32_t kW4Rows = 128;                 // rows per tile at most
constexpr uint32_t kMaxW4Jobs = 8;
constexpr uint32_t kMaxW4Tokens = 32;
constexpr uint32_t kMaxW4Cols = 1u << 24;
constexpr uint32_t kMaxW4Matrix = 0x7FFFFF00u;    // rows: tensor-map coordinates are 32-bit signed
constexpr uint32_t kMaxW4Split = 8;

enum : int { kCodesInt = 0, kCodesZero = 1, kCodesTable = 2 };

// TOK: the most tokens (2, 8, 16 or 32).
template <int CODES, int GB, int TOK>
struct W4Shape {
    static constexpr uint32_t kN = TOK <= 16 ? 16 : 32;      // MMA N
    // Columns per slab.  256 halve the waits per column, but only three stages of them fit tensor memory, and two
    // where a slab has more or wider accumulators.  28672 x 8192 at 256 and at 128 columns: groups of 128 with zero
    // points, eight tokens 36.2 and 41.4 us, 32 tokens 78.4 and 66.6; groups of 64, one token 43.9 and 37.7.
    static constexpr uint32_t kSlab = GB == 4 && TOK <= 16 ? 256 : 128;
    static constexpr uint32_t kRowBytes = kSlab / 2;         // a row's codes
    static constexpr uint32_t kCodes = kW4Rows * kRowBytes;  // a slab's, in the ring
    static constexpr uint32_t kACols = kSlab / 2;            // tensor-memory columns of a decoded slab
    static constexpr int kGroups = (int)kSlab / (32 * GB);   // groups per slab
    // Stages and groups of decoders.  32 tokens: the totals take the registers, and with groups of 32 columns the
    // accumulators the tensor memory.  Five and six stages of 128 columns measured like four.  At four stages
    // (80 registers) groups of 32 spill 24 to 32 bytes with 8 tokens and 8 with 16; with 32 tokens table codes
    // spill 80 there, zero points 8 in groups of 64.
    static constexpr uint32_t kParts = kSlab == 256 ? 3 : TOK <= 16 ? 4 : GB > 1 ? 3 : 2;
    static constexpr uint32_t kThreads = kParts * 160 + 32;
    static constexpr uint32_t kRing = 12 * 128 / kSlab;      // slabs of codes
    static constexpr uint32_t kB = kN * kSlab * 2;           // token tile of a stage
    static constexpr uint32_t kLut = CODES == kCodesTable ? 256 * 128 : 0;  // byte -> two values, one copy per bank
    static constexpr uint32_t kSums = kParts * TOK * (kW4Rows + kMaxW4Split) * 4;
    static constexpr uint32_t kSmem = 1024 + kRing * kCodes + kParts * kB + kLut + kSums;
    static_assert(kSmem <= 225 * 1024, "shared memory per block");
    // Nor room beside it for a block of eq_gemm_a8 (111 KB and more): two kernels of different streams, each with
    // clusters that wait for tensor memory the other's hold, would never end.
    static_assert(kSmem > (228 - 111 - 2) * 1024, "a second block fits");
    static constexpr uint32_t kInstrDesc = (1u << 4) | (1u << 7) | (1u << 10)  // fp32 D, bf16 A and B, K-major
                                         | ((kN >> 3) << 17) | ((kW4Rows >> 4) << 24);
    static_assert(kParts * (kACols + kGroups * kN) <= 512, "tensor memory columns");
};

struct W4Job {
    CUtensorMap tmap_q;  // uint8 [rows, cols / 2], box kRowBytes x tile rows, swizzle of that width
    const void *scales;
    const uint8_t *zeros;
    const uint16_t *x;
    float *y;
    uint64_t x_stride;
    uint32_t rows, cols, groups, scale_type;
    uint32_t first_unit;
    uint32_t pad;
    uint16_t table[16];
};

struct W4Params {
    uint32_t tokens, n_jobs, units, tile_rows;
    W4Job jobs[kMaxW4Jobs];
};
static_assert(sizeof(W4Params) <= 4096, "kernel parameter space");

__device__ __forceinline__ uint32_t sub_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t permute(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// (w & 0x000F000F) | k128: two codes as bf16(128 + q); one logic instruction, with k128 = 0x43004300
// in a register (it takes one literal only).
__device__ __forceinline__ uint32_t codes_at_128(uint32_t w, uint32_t k128) {
    uint32_t r;
    asm("lop3.b32 %0, %1, 0x000F000F, %2, 0xEA;" : "=r"(r) : "r"(w), "r"(k128));
    return r;
}

// The 8 codes of a word as four bf16 pairs.  Codes i and i + 4 sit 16 bits
// apart: under the exponent of 128 they read 128 + q, and subtracting 128 + zero
// is exact.  The shifts are high products, which run on the multiply pipe while
// the masks fill the logic pipe.  Table: byte i (codes 2 i and 2 i + 1) indexes
// the lane's own copy of the pair table, so the 32 lanes never share a bank.
template <int CODES>
__device__ __forceinline__ void decode8(uint32_t w, uint32_t zero, uint32_t k128, uint32_t lut, uint32_t *p) {
    if constexpr (CODES == kCodesTable) {
        p[0] = lds_u32(lut + ((w << 7) & 0x7F80u));
        p[1] = lds_u32(lut + (mad_hi(w, 1u << 31, 0u) & 0x7F80u));
        p[2] = lds_u32(lut + (mad_hi(w, 1u << 23, 0u) & 0x7F80u));
        p[3] = lds_u32(lut + (mad_hi(w, 1u << 15, 0u) & 0x7F80u));
    } else {
        p[0] = sub_bf16x2(codes_at_128(w, k128), zero);
        p[1] = sub_bf16x2(codes_at_128(mad_hi(w, 1u << 28, 0u), k128), zero);
        p[2] = sub_bf16x2(codes_at_128(mad_hi(w, 1u << 24, 0u), k128), zero);
        p[3] = sub_bf16x2(codes_at_128(mad_hi(w, 1u << 20, 0u), k128), zero);
    }
}

// N consecutive scales' bits (or zero points) of a row: one access where every row's are aligned to it.
template <int N>
__device__ __forceinline__ void load_scales(const void *p, uint64_t at, uint32_t type, bool vec, uint32_t in, uint32_t *v) {
    if (vec) {
        if (type == EQ_F32) {
            const uint32_t *q = static_cast<const uint32_t *>(p) + at;
            if constexpr (N == 4) {
                const uint4 w = *reinterpret_cast<const uint4 *>(q);
                v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
            } else if constexpr (N == 2) {
                const uint2 w = *reinterpret_cast<const uint2 *>(q);
                v[0] = w.x, v[1] = w.y;
            } else {
                v[0] = *q;
            }
        } else {  // two to a word: unpacked by scale_value's caller
            const uint16_t *q = static_cast<const uint16_t *>(p) + at;
            if constexpr (N == 4) {
                const uint2 w = *reinterpret_cast<const uint2 *>(q);
                v[0] = w.x, v[2] = w.y;
            } else if constexpr (N == 2) {
                v[0] = *reinterpret_cast<const uint32_t *>(q);
            } else {
                v[0] = *q;
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < (int)in)
            v[j] = type == EQ_F32 ? static_cast<const uint32_t *>(p)[at + j] : static_cast<const uint16_t *>(p)[at + j];
}

template <int N>
__device__ __forceinline__ uint32_t load_zeros(const uint8_t *p, bool vec, uint32_t in) {
    if (vec) {
        if constexpr (N == 4) return *reinterpret_cast<const uint32_t *>(p);
        if constexpr (N == 2) return *reinterpret_cast<const uint16_t *>(p);
        return *p;
    }
    uint32_t v = 0;
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (j < (int)in) v |= (uint32_t)p[j] << (8 * j);
    return v;
}

// The value of a scale's bits (apart from the load, so that it is not waited for where it is issued).
__device__ __forceinline__ float scale_value(uint32_t bits, uint32_t type) {
    return type == EQ_F32    ? __uint_as_float(bits)
           : type == EQ_BF16 ? __uint_as_float(bits << 16)
                             : __half2float(__ushort_as_half((uint16_t)bits));
}

// TOK consecutive accumulator columns of this thread's lane.
template <int TOK>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[TOK]) {
    if constexpr (TOK == 2) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    } else if constexpr (TOK == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    } else if constexpr (TOK == 16) {
        tmem_ld16(taddr, r);
    } else {
        tmem_ld32(taddr, r);
    }
}

// A tile: rows of one job.
struct W4Tile {
    uint32_t job, row0, rows;
};

__device__ __forceinline__ void tile_of(const W4Params &P, uint32_t unit, W4Tile &t) {
    while (t.job + 1 < P.n_jobs && unit >= P.jobs[t.job + 1].first_unit) ++t.job;
    const W4Job &J = P.jobs[t.job];
    t.row0 = (unit - J.first_unit) * P.tile_rows;
    t.rows = min(P.tile_rows, J.rows - t.row0);
}

// CODES: what a code means.  GB: 32-column blocks per group (group / 32).  TOK: the most tokens.
template <int CODES, int GB, int TOK>
__global__ void __launch_bounds__(W4Shape<CODES, GB, TOK>::kThreads, 1)
    eq_gemv_w4_kernel(const __grid_constant__ W4Params P) {
    using S = W4Shape<CODES, GB, TOK>;
    constexpr uint32_t kParts = S::kParts, kRing = S::kRing, kN = S::kN;
    constexpr uint32_t kSlab = S::kSlab, kACols = S::kACols, kCodes = S::kCodes;
    constexpr int NG = S::kGroups;
    constexpr uint32_t kDecoders = kParts * 4;  // warps
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t landed_s[kRing], read_s[kRing], ready_s[kParts], done_s[kParts];
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile uint32_t abort_s;
    const uint32_t tid = threadIdx.x, warp = warp_index(), lane = tid & 31u;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t btile = base, ring = btile + kParts * S::kB, lut = ring + kRing * kCodes, sums = lut + S::kLut;
    const uint32_t landed = smem_u32(&landed_s[0]), read = smem_u32(&read_s[0]);
    const uint32_t ready = smem_u32(&ready_s[0]), done = smem_u32(&done_s[0]);
    const uint32_t split = cluster_size(), rank = cluster_rank();
    const uint32_t T = P.tokens, first = blockIdx.x / split, step = gridDim.x / split;

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&tmem_base_s)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 32) {
        for (uint32_t i = 0; i < kRing; ++i) {
            mbar_init(landed + 8 * i, 1);
            mbar_init(read + 8 * i, 4);  // a group's four warps
        }
        for (uint32_t i = 0; i < kParts; ++i) {
            mbar_init(ready + 8 * i, 4);
            mbar_init(done + 8 * i, 1);
        }
        fence_mbar_init();
        abort_s = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    next_kernel_may_start();  // tensor memory is allocated
    // the cluster's CTAs have all started (waited for before the first remote store)
    if (split > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    previous_kernel_done();
    const uint32_t tmem = tmem_base_s;
    const uint32_t acc0 = tmem + kParts * kACols;  // accumulators: [stage][group][token]
    bool ok = true;
    // this CTA's slabs of a tile
    const auto slab_range = [&](uint32_t cols, uint32_t &k0, uint32_t &k1) {
        const uint32_t slabs = (cols + kSlab - 1) / kSlab;
        k0 = slabs * rank / split, k1 = slabs * (rank + 1) / split;
    };

    if (warp < kDecoders) {
        // ---- decoders ----
        const uint32_t part = warp >> 2, quarter = warp & 3u, row = quarter * 32u + lane;
        const uint32_t lane_base = (quarter * 32u) << 16;
        const uint32_t ta = tmem + lane_base + part * kACols, td = acc0 + lane_base + part * (NG * kN);
        const uint32_t my_lut = lut + lane * 4;
        uint32_t k128;
        asm volatile("mov.b32 %0, 0x43004300;" : "=r"(k128));
        {  // rows that no tile fills are products too: never of unwritten memory
            uint32_t zero[16] = {};
#pragma unroll
            for (uint32_t c = 0; c < kACols; c += 16) tmem_st16(ta + c, zero);
            tmem_st_wait();
        }
        uint32_t g0 = 0, uses = 0, lut_job = 0xFFFFFFFFu;  // slabs before this tile; this group's slabs so far
        W4Tile t{0, 0, 0};
        for (uint32_t unit = first; unit < P.units; unit += step) {
            if (__any_sync(0xFFFFFFFFu, abort_s != 0u)) ok = false;
            tile_of(P, unit, t);
            const W4Job &J = P.jobs[t.job];
            const uint32_t type = J.scale_type, groups = J.groups;
            uint32_t k0, k1;
            slab_range(J.cols, k0, k1);
            if constexpr (CODES == kCodesTable) {
                if (lut_job != t.job) {  // byte b's two values, in all 32 banks
                    lut_job = t.job;
                    asm volatile("bar.sync 1, %0;" ::"r"(kDecoders * 32) : "memory");
                    if (tid < 256) {
                        const uint32_t v = (uint32_t)J.table[tid & 15u] | (uint32_t)J.table[tid >> 4] << 16;
#pragma unroll
                        for (uint32_t i = 0; i < 8; ++i)
                            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                             lut + tid * 128 + ((i + tid) & 7u) * 16),
                                         "r"(v)
                                         : "memory");
                    }
                    asm volatile("bar.sync 1, %0;" ::"r"(kDecoders * 32) : "memory");
                }
            }
            const bool mine = row < t.rows;                 // this thread's row exists
            const bool busy = quarter * 32u < t.rows;       // ... or another of the warp's
            const uint64_t srow = (uint64_t)(t.row0 + row) * groups;
            // one access per slab where every row's groups are a whole number of slabs (and aligned)
            const uint32_t size = type == EQ_F32 ? 4 : 2;
            const bool s_vec = groups % NG == 0 && reinterpret_cast<uintptr_t>(J.scales) % (NG * size) == 0;
            const bool z_vec = CODES == kCodesZero && groups % NG == 0 && reinterpret_cast<uintptr_t>(J.zeros) % NG == 0;
            uint32_t s_raw[NG], z_raw = 0;
            const auto fetch = [&](uint32_t k) {
                const uint32_t in = mine ? min((uint32_t)NG, groups - k * NG) : 0;
#pragma unroll
                for (int j = 0; j < NG; ++j) s_raw[j] = 0;
                if (in == 0) return;
                load_scales<NG>(J.scales, srow + k * NG, type, s_vec, in, s_raw);
                if constexpr (CODES == kCodesZero) z_raw = load_zeros<NG>(J.zeros + srow + k * NG, z_vec, in);
            };
            float total[TOK];
#pragma unroll
            for (int i = 0; i < TOK; ++i) total[i] = 0.f;
            float s[NG];
            bool pending = false;
            const auto drain = [&]() {  // the last slab's sums
                if (!warp_wait(done + 8 * part, (uses - 1) & 1u)) {
                    ok = false;
                    return;
                }
                tc_fence_after();
                if (busy) {
#pragma unroll
                    for (int j = 0; j < NG; ++j) {
                        uint32_t acc[TOK];
                        tmem_ld<TOK>(td + j * kN, acc);
#pragma unroll
                        for (int i = 0; i < TOK; ++i) total[i] = fmaf(s[j], __uint_as_float(acc[i]), total[i]);
                    }
                }
            };
            uint32_t k = k0 + part;
            if (k < k1) fetch(k);
            uint32_t slot = (g0 + part) % kRing, lap = (g0 + part) / kRing & 1u;
            // the first 16 bytes of this row in slot 0; block c's are at exclusive or 16 c (64- or 128-byte swizzle)
            const uint32_t row_at = ring + row * S::kRowBytes + (kSlab == 256 ? (row & 7u) << 4 : ((row >> 1) & 3u) << 4);
            for (; k < k1 && ok; k += kParts) {
                float s_now[NG];
                uint32_t zero[NG];
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                    uint32_t bits = s_raw[j];
                    if (NG > 1 && s_vec && size == 2) bits = (s_raw[j & ~1] >> (16 * (j & 1))) & 0xFFFFu;
                    s_now[j] = scale_value(bits, type);
                    zero[j] = 0x43084308u;
                    if constexpr (CODES == kCodesZero) {  // bf16(128 + zero) is exact up to 127; more marks the sums
                        zero[j] = 0x43004300u | (z_raw >> (8 * j) & 127u) * 0x00010001u;
                        if (z_raw >> (8 * j) & 128u) s_now[j] = __uint_as_float(0x7FC00000u);
                    }
                }
                if (k + kParts < k1) fetch(k + kParts);
                if (!warp_wait(landed + 8 * slot, lap)) {
                    ok = false;
                    break;
                }
                // the first kAhead of the slab's 32-column blocks are decoded before the last slab's
                // products are waited for, so that decoding covers their latency
                constexpr uint32_t kAhead = TOK <= 8 ? 2 : 1;
                const uint32_t from = row_at + slot * kCodes;
                const auto decode_block = [&](uint32_t c, uint32_t *p) {
                    uint32_t w[4];
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]),
                                 "=r"(w[3]) : "r"(from ^ (c << 4)));
#pragma unroll
                    for (int i = 0; i < 4; ++i) decode8<CODES>(w[i], zero[c / GB], k128, my_lut, p + 4 * i);
                };
                uint32_t ahead[kAhead][16];
                if (busy) {
#pragma unroll
                    for (uint32_t c = 0; c < kAhead; ++c) decode_block(c, ahead[c]);
                }
                if (pending) drain();
                if (!ok) break;
                if (busy) {
#pragma unroll
                    for (uint32_t c = 0; c < kAhead; ++c) tmem_st16(ta + c * 16, ahead[c]);
#pragma unroll
                    for (uint32_t c = kAhead; c < kSlab / 32; ++c) {
                        uint32_t p[16];
                        decode_block(c, p);
                        tmem_st16(ta + c * 16, p);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                warp_arrive(ready + 8 * part);
                warp_arrive(read + 8 * slot);
#pragma unroll
                for (int j = 0; j < NG; ++j) s[j] = s_now[j];
                slot += kParts;
                if (slot >= kRing) slot -= kRing, lap ^= 1u;
                ++uses;
                pending = true;
            }
            if (ok && pending) drain();
            g0 += k1 - k0;
            // the totals of the groups (and of the cluster's CTAs): CTA q owns rows [q R, (q + 1) R) of the
            // tile, source (CTA, group) is at [source][token][row]
            const uint32_t R = (kW4Rows + split - 1) / split, src = rank * kParts + part;
            const uint32_t owner = row / R, local = row - owner * R;
            if (split > 1)
                asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
            else
                asm volatile("bar.sync 1, %0;" ::"r"(kDecoders * 32) : "memory");  // the last tile's have been read
            const uint32_t to = cluster_addr(sums + (src * T * R + local) * 4, owner);
#pragma unroll
            for (int i = 0; i < TOK; ++i)
                if (i < (int)T)
                    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + i * R * 4),
                                 "f"(ok ? total[i] : __uint_as_float(0x7FC00000u))
                                 : "memory");
            if (split > 1) break;  // one tile per cluster; its sums follow below
            asm volatile("bar.sync 1, %0;" ::"r"(kDecoders * 32) : "memory");
            for (uint32_t e = tid; e < T * kW4Rows; e += kDecoders * 32) {
                const uint32_t tok = e / kW4Rows, r = e % kW4Rows;
                if (r >= t.rows) continue;
                float v = 0.f;
#pragma unroll
                for (uint32_t q = 0; q < kParts; ++q)
                    v = __fadd_rn(v, __uint_as_float(lds_u32(sums + ((q * T + tok) * kW4Rows + r) * 4)));
                J.y[(uint64_t)tok * J.rows + t.row0 + r] = v;
            }
        }
    } else if (warp < kDecoders + kParts) {
        // ---- products (converged warps, one lane of which issues) ----
        constexpr uint32_t kChunks = kSlab / 8, kTokStep = 32 / kChunks;  // a lane: 8 columns of every kTokStep-th token
        constexpr int kVecs = TOK / kTokStep;
        const uint32_t part = warp - kDecoders, chunk = lane % kChunks, tok0 = lane / kChunks;
        const uint32_t d = acc0 + part * (NG * kN), ta = tmem + part * kACols;
        const uint64_t b0 = smem_desc(btile + part * S::kB, 16u, 1024u);
        uint32_t ph = 0;  // the parity of the stage's next use
        bool again = false;
        W4Tile t{0, 0, 0};
        for (uint32_t unit = first; unit < P.units && ok; unit += step) {
            tile_of(P, unit, t);
            const W4Job &J = P.jobs[t.job];
            uint32_t k0, k1;
            slab_range(J.cols, k0, k1);
            const uint16_t *x0 = J.x + tok0 * J.x_stride + chunk * 8;
            uint4 v[kVecs];
            const auto fetch = [&](uint32_t k) {
                const bool in = k * kSlab + chunk * 8 < J.cols;
#pragma unroll
                for (int i = 0; i < kVecs; ++i)
                    v[i] = in && tok0 + kTokStep * i < T
                               ? *reinterpret_cast<const uint4 *>(x0 + kTokStep * i * J.x_stride + k * kSlab)
                               : make_uint4(0, 0, 0, 0);
            };
            uint32_t k = k0 + part;
            if (k < k1) fetch(k);
            for (; k < k1; k += kParts) {
                if (again && !warp_wait(done + 8 * part, ph ^ 1u)) {
                    ok = false;
                    break;
                }
                // K-major, 128-byte swizzle: columns 64 (chunk / 8) + 8 (chunk % 8) .. + 7 of token n
                const uint32_t dst = btile + part * S::kB + (chunk >> 3) * (kN * 128);
#pragma unroll
                for (int i = 0; i < kVecs; ++i) {
                    const uint32_t n = tok0 + kTokStep * i;
                    uint4 o = v[i];
                    if constexpr (CODES != kCodesTable) {  // pair columns i and i + 4
                        o.x = permute(v[i].x, v[i].z, 0x5410u);
                        o.y = permute(v[i].x, v[i].z, 0x7632u);
                        o.z = permute(v[i].y, v[i].w, 0x5410u);
                        o.w = permute(v[i].y, v[i].w, 0x7632u);
                    }
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     dst + n * 128 + (((chunk & 7u) ^ (n & 7u)) << 4)),
                                 "r"(o.x), "r"(o.y), "r"(o.z), "r"(o.w)
                                 : "memory");
                }
                if (k + kParts < k1) fetch(k + kParts);
                fence_proxy_async_smem();
                __syncwarp();
                if (!warp_wait(ready + 8 * part, ph)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (uint32_t j = 0; j < kSlab / 16; ++j)  // 16 columns: 32 bytes of B in one of its 64-column atoms
                        tc_mma_ts(d + (j / (2 * GB)) * kN, ta + j * 8, b0 + (((j >> 2) * (kN * 128) + (j & 3u) * 32) >> 4),
                                  S::kInstrDesc, j % (2 * GB) != 0);
                    tc_commit(done + 8 * part);
                }
                __syncwarp();
                ph ^= 1u;
                again = true;
            }
        }
    } else {
        // ---- loader (a converged warp, one lane of which copies) ----
        uint32_t g = 0, slot = 0, ph = 0;
        W4Tile t{0, 0, 0};
        const uint32_t bytes = P.tile_rows * S::kRowBytes;
        for (uint32_t unit = first; unit < P.units && ok; unit += step) {
            tile_of(P, unit, t);
            const W4Job &J = P.jobs[t.job];
            uint32_t k0, k1;
            slab_range(J.cols, k0, k1);
            for (uint32_t k = k0; k < k1; ++k, ++g) {
                if (g >= kRing && !warp_wait(read + 8 * slot, ph ^ 1u)) {
                    ok = false;
                    break;
                }
                const uint32_t bar = landed + 8 * slot;
                if (elect_one()) {
                    mbar_expect_tx(bar, bytes);
                    tma_2d(ring + slot * kCodes, &J.tmap_q, k * S::kRowBytes, t.row0, bar);
                }
                __syncwarp();
                if (++slot == kRing) {
                    slot = 0;
                    ph ^= 1u;
                }
            }
        }
        // no copy may still be writing shared memory when the CTA leaves
        for (uint32_t k = g > kRing ? g - kRing : 0; k < g; ++k)
            if (!warp_wait(landed + 8 * (k % kRing), (k / kRing) & 1u)) ok = false;
    }
    if (!ok) abort_s = 1;
    __syncwarp();
    if (split > 1) {
        if (warp >= kDecoders) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
        __syncwarp();
        cluster_sync_all();
        W4Tile t{0, 0, 0};
        tile_of(P, first, t);
        const W4Job &J = P.jobs[t.job];
        const uint32_t R = (kW4Rows + split - 1) / split;
        for (uint32_t e = tid; e < T * R; e += S::kThreads) {
            const uint32_t tok = e / R, local = e - tok * R, r = rank * R + local;
            if (r >= t.rows) continue;
            float v = 0.f;
            for (uint32_t src = 0; src < split * kParts; ++src)
                v = __fadd_rn(v, __uint_as_float(lds_u32(sums + ((src * T + tok) * R + local) * 4)));
            J.y[(uint64_t)tok * J.rows + t.row0 + r] = v;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

int encode_code_map(CUtensorMap *map, const void *q, uint32_t rows, uint32_t cols, uint32_t slab, uint32_t box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return EQ_ERR_CUDA;
    const cuuint64_t dims[2] = {cols / 2, rows};
    const cuuint64_t strides[1] = {cols / 2};
    const cuuint32_t box[2] = {slab / 2, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(q), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE,
                           slab == 256 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? EQ_OK : EQ_ERR_CUDA;
}

struct W4Kernel {
    const void *fn;
    uint32_t smem, threads, slab;
};

template <int CODES, int GB, int TOK>
W4Kernel w4_kernel() {
    using S = W4Shape<CODES, GB, TOK>;
    return {(const void *)eq_gemv_w4_kernel<CODES, GB, TOK>, S::kSmem, S::kThreads, S::kSlab};
}

template <int CODES, int GB>
W4Kernel pick_tokens(uint32_t tokens) {
    return tokens <= 2    ? w4_kernel<CODES, GB, 2>()
           : tokens <= 8  ? w4_kernel<CODES, GB, 8>()
           : tokens <= 16 ? w4_kernel<CODES, GB, 16>()
                          : w4_kernel<CODES, GB, 32>();
}

template <int CODES>
W4Kernel pick_group(uint32_t group, uint32_t tokens) {
    return group == 32 ? pick_tokens<CODES, 1>(tokens)
                       : group == 64 ? pick_tokens<CODES, 2>(tokens) : pick_tokens<CODES, 4>(tokens);
}

int codes_of(const eq_w4_job &j) { return j.use_table ? kCodesTable : j.zeros ? kCodesZero : kCodesInt; }

int check_w4(const eq_w4_job &j, uint32_t tokens) {
    if (j.scale_type != EQ_F32 && j.scale_type != EQ_BF16 && j.scale_type != EQ_F16) return EQ_ERR_INVALID_ARG;
    if (j.use_table > 1 || (j.use_table && j.zeros)) return EQ_ERR_INVALID_ARG;
    if (j.use_table)  // the code of a missing row or column may be any
        for (uint16_t v : j.table)
            if ((v & 0x7F80u) == 0x7F80u) return EQ_ERR_INVALID_ARG;
    if (!j.rows) return EQ_OK;
    if (j.rows > kMaxW4Matrix) return EQ_ERR_UNSUPPORTED;
    if (!j.cols || j.cols % 32 || j.cols > kMaxW4Cols || (j.group != 32 && j.group != 64 && j.group != 128))
        return EQ_ERR_UNSUPPORTED;
    if (!j.q || !j.scales || (tokens && (!j.x || !j.y))) return EQ_ERR_INVALID_ARG;
    const auto at = [](const void *p) { return reinterpret_cast<uintptr_t>(p); };
    if (at(j.q) % 16 || at(j.x) % 16 || at(j.y) % 4 || at(j.scales) % (j.scale_type == EQ_F32 ? 4 : 2))
        return EQ_ERR_INVALID_ARG;
    if (tokens > 1 && (j.x_stride < j.cols || j.x_stride % 8)) return EQ_ERR_INVALID_ARG;
    return EQ_OK;
}

// How many clusters of `split` CTAs with a whole SM each run at once on device `dev`.  Asked once.
uint32_t resident_clusters(int dev, uint32_t split, const W4Kernel &kn, uint32_t sms) {
    static std::atomic<uint32_t> known[128][kMaxW4Split + 1];
    std::atomic<uint32_t> &slot = known[dev][split];
    uint32_t n = slot.load(std::memory_order_relaxed);
    if (n) return n;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(split);
    cfg.blockDim = dim3(kn.threads);
    cfg.dynamicSmemBytes = kn.smem;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = split;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int got = 0;
    if (cudaOccupancyMaxActiveClusters(&got, kn.fn, &cfg) != cudaSuccess || got <= 0) {
        (void)cudaGetLastError();
        return sms / split;
    }
    n = std::min<uint32_t>((uint32_t)got, sms / split);
    slot.store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace

extern "C" EQW_API int eq_gemv_w4(const eq_w4_job *jobs, uint32_t n_jobs, uint32_t tokens, cudaStream_t s) try {
    const eqw::NvtxScope nvtx_range("eq_gemv_w4");
    if (n_jobs && !jobs) return EQ_ERR_INVALID_ARG;
    for (uint32_t i = 0; i < n_jobs; ++i)
        if (const int rc = check_w4(jobs[i], tokens)) return rc;
    if (tokens > kMaxW4Tokens) return EQ_ERR_UNSUPPORTED;
    std::vector<const eq_w4_job *> live;
    for (uint32_t i = 0; i < n_jobs; ++i)
        if (jobs[i].rows) live.push_back(&jobs[i]);
    if (!tokens || live.empty()) return EQ_OK;
    // jobs of one code form and group size share a launch
    std::stable_sort(live.begin(), live.end(), [](const eq_w4_job *a, const eq_w4_job *b) {
        const int ca = codes_of(*a), cb = codes_of(*b);
        return ca != cb ? ca < cb : a->group != b->group ? a->group < b->group : a->cols > b->cols;
    });
    int dev = 0, sm_count = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 128 ||
        cudaDeviceGetAttribute(&sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sm_count <= 0)
        return EQ_ERR_CUDA;
    const uint32_t sms = (uint32_t)sm_count;
    for (size_t at = 0; at < live.size();) {
        const int codes = codes_of(*live[at]);
        const uint32_t group = live[at]->group;
        const W4Kernel kn = codes == kCodesInt    ? pick_group<kCodesInt>(group, tokens)
                            : codes == kCodesZero ? pick_group<kCodesZero>(group, tokens)
                                                  : pick_group<kCodesTable>(group, tokens);
        if (cudaFuncSetAttribute(kn.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kn.smem) != cudaSuccess)
            return EQ_ERR_CUDA;
        size_t end = at;
        while (end < live.size() && end - at < kMaxW4Jobs && codes_of(*live[end]) == codes && live[end]->group == group)
            ++end;
        const auto tiles = [&](uint32_t rows) {
            uint64_t n = 0;
            for (size_t k = at; k < end; ++k) n += ((uint64_t)live[k]->rows + rows - 1) / rows;
            return n;
        };
        uint32_t min_slabs = 0xFFFFFFFFu;
        for (size_t k = at; k < end; ++k) min_slabs = std::min(min_slabs, (live[k]->cols + kn.slab - 1) / kn.slab);
        // Whole tiles fill the SMs: as many rounds as 128-row tiles take, with tiles of equal height.  Fewer
        // tiles than SMs: the CTAs of a cluster share K, each keeping at least 512 columns, and the tiles get lower
        // (not below a warp's 32 rows) until the clusters fill the SMs.
        const uint64_t full = tiles(kW4Rows);
        uint32_t split = 1;
        uint64_t room = (full + sms - 1) / sms * sms;
        if (full < sms) {
            split = std::max(1u, std::min({kMaxW4Split, (uint32_t)(sms / full), min_slabs * kn.slab / 512}));
            while (split > 1 && resident_clusters(dev, split, kn, sms) < full) --split;
            room = split > 1 ? resident_clusters(dev, split, kn, sms) : sms;
        }
        uint32_t rows = 32;
        while (rows < kW4Rows && tiles(rows) > room) ++rows;
        W4Params P{};
        P.tokens = tokens;
        P.tile_rows = rows;
        const uint64_t units = tiles(rows);
        if (units > 0x0FFFFFFFull) return EQ_ERR_UNSUPPORTED;
        P.units = (uint32_t)units;
        uint32_t unit = 0;
        for (; at < end; ++at) {
            const eq_w4_job &q = *live[at];
            W4Job &J = P.jobs[P.n_jobs++];
            if (const int rc = encode_code_map(&J.tmap_q, q.q, q.rows, q.cols, kn.slab, rows)) return rc;
            J.scales = q.scales, J.zeros = q.zeros, J.x = static_cast<const uint16_t *>(q.x), J.y = q.y;
            J.x_stride = tokens > 1 ? q.x_stride : 0;
            J.rows = q.rows, J.cols = q.cols, J.groups = (q.cols + group - 1) / group, J.scale_type = q.scale_type;
            std::memcpy(J.table, q.table, sizeof(J.table));
            J.first_unit = unit;
            unit += (q.rows + rows - 1) / rows;
        }
        void *args[] = {&P};
        const uint32_t grid = split > 1 ? (uint32_t)units * split : (uint32_t)std::min<uint64_t>(units, sms);
        if (!launch_overlapped(kn.fn, grid, kn.threads, kn.smem, split, args, s)) return EQ_ERR_CUDA;
    }
    return EQ_OK;
} catch (...) {  // host memory for the job list
    return EQ_ERR_NOSPACE;
}
