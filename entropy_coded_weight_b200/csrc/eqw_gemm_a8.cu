// 8-bit tokens times 8-bit weight symbols on the 5th-generation tensor cores:
// eq_gemm_a8, eq_gemm_symbols_a8, eq_gemm_symbols_a8_block.
//
//   Y[t, r] = ws[r] * (xs[t] * S[t, r]),   S[t, r] = sum_c x8[t, c] * sym[r, c]
//             + sum over super weights (r, c, v) of bf16(v) * xs[t] * x8[t, c]
// x8 and sym are both Int8 (kind::i8: S is exact in int32, which bounds cols)
// or both E4M3 (kind::f8f6f4, fp32 accumulator).  Both operands go from HBM to
// the tensor core unwidened: TMA copies (128-byte swizzle, K-major) into
// shared memory, tcgen05.mma with M = weight rows, N = tokens, K = 32, the
// accumulator in tensor memory (lane = weight row, column = token).
//
// Two kernels, chosen per launch by the host:
//   eq_gemm_a8_split_kernel  128 weight rows x up to 256 tokens per cluster of
//                            CTAs that split K between them; the partial sums
//                            meet over distributed shared memory in a fixed order
//   eq_gemm_a8_pair_kernel   256 x 256 tiles on pairs of SMs (cta_group::2),
//                            persistent, two accumulators so that a tile's
//                            epilogue runs beside the next tile's products
// Super weights are added by the CTA that wrote their outputs, after its stores.
//
// Measured (B200, launches back to back on rotating inputs larger than L2): few
// tokens are bound by memory, one Int8 token x 8192 x 8192 in 14.1 us (4.8 TB/s; about
// 3 us are launch, first copies and the exchange of sums), 48 E4M3 tokens x 28672 x
// 8192 in 40 us (5.9 TB/s).  Many are bound by the tensor cores and their power:
// 4096 tokens x 28672 x 8192 in 626 to 667 us Int8 (2.9 to 3.1 POP/s, tensor pipe 93 %
// of active clocks) and 750 to 850 us E4M3 (2.3 to 2.6 PFLOP/s at a lower clock).
#include <cuda.h>
#include <cuda_runtime.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <vector>

#include "eqw_device.cuh"
#include "eqw_launch.cuh"
#include "eqw_tc.cuh"

namespace {

constexpr uint32_t kRowsTile = 128;                      // weight rows per CTA (accumulator lanes)
constexpr uint32_t kSlab = 128;                          // K per stage: one 128-byte swizzle row
constexpr uint32_t kMmaK8 = 32;                          // K per tcgen05.mma on 8-bit types
constexpr uint32_t kAtom = 8 * kSlab;                    // 8-row swizzle atom (SBO)
constexpr uint32_t kWTile = kRowsTile * kSlab;           // 16 KB of symbols per stage
constexpr uint32_t kMaxA8Jobs = 8;  // (kernel parameters: 4 KB)
constexpr uint32_t kA8Threads = 192;                     // split: 4 epilogue warps, the loader warp, the MMA warp
constexpr uint32_t kPairThreads = 320;                   // pairs: 8 epilogue warps, the loader warp, the MMA warp
constexpr uint32_t kPairEpilogue = 256;                  // their threads
constexpr uint32_t kMaxSplit = 8;
constexpr uint32_t kMaxRows = 0x7FFFFF00u;               // (and columns) tensor-map coordinates are 32-bit signed
constexpr uint32_t kMaxInt8Cols = 131056;                // 128 * 128 * cols < 2^31
// E4M3: the tensor core rounds its accumulator towards zero at every step, so a chain's error is a bias that grows
// with its length. Relative to the result's norm, one accumulator for all of K: 2.3e-7 at 32 slabs, 5.0e-7 at 64, 2.5e-6
// at 224; fp32 products summed in order by a library: 0.9e-7, 1.3e-7, 2.8e-7. So K is cut into chains with an
// accumulator each, whose values are added in fp32, rounded to nearest: with chains of 16 slabs 1.2e-7 to 1.4e-7 at
// any K. A split CTA that has no tensor memory for as many accumulators takes chains of up to twice that.
constexpr uint32_t kChain = 16;

// Instruction descriptor: 8-bit K-major operands, N tokens, M rows.
template <int DT>
__host__ __device__ constexpr uint32_t instr_desc(uint32_t n, uint32_t m) {
    return (DT == EQ_INT8 ? (2u << 4) | (1u << 7) | (1u << 10)  // int32 accumulator, signed A and B
                          : (1u << 4))                          // fp32 accumulator, E4M3 (0) A and B
           | ((n >> 3) << 17) | ((m >> 4) << 24);
}

constexpr uint32_t kMaxStages = 8;
constexpr uint32_t kSplitTok = 256;                      // most tokens of a split tile
constexpr size_t kSplitSmem2 = 111 * 1024;               // dynamic shared memory with two CTAs per SM ...
constexpr size_t kSplitSmem1 = 224 * 1024;               // ... and with one

struct A8Job {
    CUtensorMap tmap_w;  // uint8 [rows, cols], box 128 bytes x 128 rows, 128-byte swizzle
    CUtensorMap tmap_x;  // uint8 [tokens, cols], box 128 bytes x the tile's tokens
    const float *ws, *xs;
    float *y;
    const uint8_t *x8;
    const uint32_t *out_row, *out_col;  // super weights, sorted by row
    const float *out_val;
    uint32_t rows, cols;
    uint32_t first_unit;
    uint32_t n_out, out_stride;
    uint32_t pad;
};

struct A8Params {
    int32_t *status;
    uint32_t tokens, t_tiles, n_jobs, total_units;
    uint32_t tok;             // split kernel: tokens per tile (a multiple of 16), its stages and their size,
    uint32_t stages, stage_bytes, tmem_cols;  // and the accumulators' columns
    uint32_t accs;            // accumulators that share a CTA's K (E4M3)
    A8Job jobs[kMaxA8Jobs];
};
static_assert(sizeof(A8Params) <= 4096, "kernel parameter space");

__device__ __forceinline__ uint64_t slab_desc(uint32_t buf) { return smem_desc(buf, 16u, kAtom); }

template <int DT>
__device__ __forceinline__ void mma8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (DT == EQ_INT8)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"(accumulate)
            : "memory");
}

// S (an int32 or fp32 bit pattern) -> Y: the token's scale, then the row's.
template <int DT>
__device__ __forceinline__ float scaled(uint32_t s, float xs, float ws) {
    const float v = DT == EQ_INT8 ? (float)(int32_t)s : __uint_as_float(s);
    return __fmul_rn(__fmul_rn(v, xs), ws);
}

// First super weight of a row >= r.
__device__ __forceinline__ uint32_t first_outlier(const A8Job &J, uint32_t r) {
    uint32_t lo = 0, hi = J.n_out;
    while (lo < hi) {
        const uint32_t mid = (lo + hi) / 2;
        if (J.out_row[(size_t)mid * J.out_stride] < r)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// Y[t, r] += sum of bf16(v) * xs[t] * x8[t, c] over the super weights of rows [n0, n0 + 128), for this CTA's
// tokens: count of them, the i-th is 4 (first + step (i / 4)) + i % 4 from m0 on, up to toks.  The epilogue's
// threads share the (row, token) pairs; each output has one writer.  The stores that wrote Y have been
// ordered before by a barrier.
template <int DT>
__device__ __noinline__ void add_outliers(const A8Job &J, uint32_t n0, uint32_t m0, uint32_t toks, uint32_t first,
                                          uint32_t step, uint32_t tid, uint32_t threads) {
    const uint32_t lo = first_outlier(J, n0), hi = first_outlier(J, n0 + kRowsTile);
    if (lo == hi) return;
    const uint32_t chunks = first * 4 < toks ? ((toks + 3) / 4 - first + step - 1) / step : 0, count = chunks * 4;
    constexpr uint32_t kMost = 1u << 20;  // entries at a time: their (entry, token) pairs have 32-bit numbers
    for (uint32_t from = lo; from < hi; from += min(hi - from, kMost)) {
        const uint32_t pairs = min(hi - from, kMost) * count;
        for (uint32_t id = tid; id < pairs; id += threads) {
            uint32_t o = from + id / count;
            const uint32_t i = id % count, c = 4 * (first + step * (i / 4)) + i % 4, t = m0 + c;
            const uint32_t r = J.out_row[(size_t)o * J.out_stride];
            // entries out of order may bring rows of other tiles here, whose outputs other CTAs write
            if (c >= toks || r >= J.rows || r - n0 >= kRowsTile) continue;
            if (o > lo && J.out_row[(size_t)(o - 1) * J.out_stride] == r) continue;  // counted with the first
            const float sc = J.xs[t];
            float sum = 0.f;
            for (; o < hi && J.out_row[(size_t)o * J.out_stride] == r; ++o) {
                const size_t at = (size_t)o * J.out_stride;
                const uint32_t col = J.out_col[at];
                if (col >= J.cols) continue;  // reported by check_outliers
                const float w = __bfloat162float(__float2bfloat16_rn(J.out_val[at]));
                sum = fmaf(w, __fmul_rn(sc, symbol_value<DT>(J.x8[(size_t)t * J.cols + col])), sum);
            }
            float *y = J.y + (size_t)t * J.rows + r;
            *y = __fadd_rn(*y, sum);
        }
    }
}

// The epilogue's warps, each as a whole.
template <int THREADS>
__device__ __forceinline__ void epilogue_sync() {
    __syncwarp();
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// Reports super weights outside their matrix or out of order: entries first, first + step, ...
__device__ __forceinline__ void check_outliers(const A8Job &J, uint32_t first, uint32_t step, int32_t *status) {
    bool bad = false;
    for (uint32_t o = first; o < J.n_out; o += step) {
        const uint32_t r = J.out_row[(size_t)o * J.out_stride];
        bad |= r >= J.rows || J.out_col[(size_t)o * J.out_stride] >= J.cols ||
               (o > 0 && J.out_row[(size_t)(o - 1) * J.out_stride] > r);
    }
    if (bad) atomicOr(status, EQ_DEV_BAD_OUTLIER);
}

template <int DT>
__global__ void __launch_bounds__(kA8Threads, 2) eq_gemm_a8_split_kernel(const __grid_constant__ A8Params P) {
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full_s[kMaxStages], empty_s[kMaxStages], done_s;
    __shared__ uint32_t tmem_base_s;
    const uint32_t tid = threadIdx.x, warp = warp_index(), lane = tid & 31u;
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t full0 = smem_u32(&full_s[0]), empty0 = smem_u32(&empty_s[0]), done = smem_u32(&done_s);
    const uint32_t stages = P.stages, stage_bytes = P.stage_bytes, TT = P.tok;
    const uint32_t parts = cluster_size(), rank = cluster_rank();
    const uint32_t unit = blockIdx.x / parts;
    uint32_t jb = 0;
    while (jb + 1 < P.n_jobs && unit >= P.jobs[jb + 1].first_unit) ++jb;
    const A8Job &J = P.jobs[jb];
    const uint32_t local = unit - J.first_unit;
    const uint32_t n0 = (local / P.t_tiles) * kRowsTile, m0 = (local % P.t_tiles) * TT;
    const uint32_t slabs = (J.cols + kSlab - 1) / kSlab;  // >= parts (host)
    const uint32_t k0 = (uint32_t)((uint64_t)slabs * rank / parts), k1 = (uint32_t)((uint64_t)slabs * (rank + 1) / parts);
    const uint32_t accs = DT == EQ_INT8 ? 1u : min(P.accs, k1 - k0);

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&tmem_base_s)), "r"(P.tmem_cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 128) {
        for (uint32_t st = 0; st < stages; ++st) {
            mbar_init(full0 + 8 * st, 1);
            mbar_init(empty0 + 8 * st, 1);
        }
        mbar_init(done, 1);
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    next_kernel_may_start();  // tensor memory is allocated
    previous_kernel_done();
    const uint32_t tmem = tmem_base_s;
    const uint32_t row = warp * 32u + lane, r = n0 + row;  // epilogue warps: accumulator lane = weight row
    float ws = 0.f;
    bool ok = true;

    if (warp == 4) {
        // ---- loader: symbol tile and token tile of each of this CTA's slabs ----
        // Row tiles start at different slabs and wrap around: in step, all of them would ask the same few
        // L2 lines for the same token tile at the same time.
        uint32_t st = 0, ph = 0, g = 0, k = k0 + (uint32_t)((uint64_t)(n0 / kRowsTile) * 5 % (k1 - k0));
        for (; g < k1 - k0; ++g, k = k + 1 == k1 ? k0 : k + 1) {
            if (g >= stages && !warp_wait(empty0 + 8 * st, ph ^ 1u)) {
                ok = false;
                break;
            }
            if (elect_one()) {
                const uint32_t buf = base + st * stage_bytes, bar = full0 + 8 * st;
                mbar_expect_tx(bar, stage_bytes);
                tma_2d(buf, &J.tmap_w, k * kSlab, n0, bar);
                tma_2d(buf + kWTile, &J.tmap_x, k * kSlab, m0, bar);
            }
            __syncwarp();
            if (++st == stages) {
                st = 0;
                ph ^= 1u;
            }
        }
        // no copy may still be writing shared memory later on
        for (uint32_t i = g > stages ? g - stages : 0; i < g; ++i)
            if (!warp_wait(full0 + 8 * (i % stages), (i / stages) & 1u)) ok = false;
    } else if (warp == 5) {
        // ---- MMA ----
        if (J.n_out && local == 0 && rank == 0) check_outliers(J, lane, 32, P.status);
        uint32_t st = 0, ph = 0;
        const uint32_t idesc = instr_desc<DT>(TT, kRowsTile);
        const uint64_t a0 = slab_desc(base), b0 = slab_desc(base + kWTile);
        uint32_t acc = 0, from = k0, to = k0 + (k1 - k0) / accs;  // this accumulator's slabs
        for (uint32_t k = k0; k < k1; ++k) {
            if (k == to) {
                ++acc;
                from = to, to = k0 + (k1 - k0) * (acc + 1) / accs;
            }
            if (!warp_wait(full0 + 8 * st, ph)) {
                ok = false;
                break;
            }
            tc_fence_after();
            if (elect_one()) {
                const uint64_t off = (uint64_t)((st * stage_bytes) >> 4);
#pragma unroll
                for (uint32_t kk = 0; kk < kSlab / kMmaK8; ++kk)  // K step: 32 bytes, 2 descriptor units
                    mma8<DT>(tmem + acc * TT, a0 + off + 2u * kk, b0 + off + 2u * kk, idesc, (k - from) | kk);
                tc_commit(empty0 + 8 * st);
                if (k + 1 == k1) tc_commit(done);
            }
            __syncwarp();
            if (++st == stages) {
                st = 0;
                ph ^= 1u;
            }
        }
        // nothing runs when the tensor memory is released
        if (!ok || !warp_wait(done, 0)) ok = false;
    } else {
        if (r < J.rows) ws = J.ws[r];
        if (!warp_wait(done, 0)) ok = false;
        tc_fence_after();
    }
    if (!ok) atomicOr(P.status, EQ_DEV_TIMEOUT);
    __syncwarp();
    const uint32_t lane_base = tmem + ((warp * 32u) << 16);
    const auto load_sums = [&](uint32_t c, uint32_t (&v)[16]) {  // 16 tokens' sums of the accumulators, in order
        __syncwarp();  // rows past the end skip what the others' lanes do with them
        tmem_ld16(lane_base + c, v);
        if constexpr (DT == EQ_E4M3) {
#pragma unroll 1
            for (uint32_t a = 1; a < accs; ++a) {
                uint32_t more[16];
                tmem_ld16(lane_base + a * TT + c, more);
#pragma unroll
                for (uint32_t j = 0; j < 16; ++j)
                    v[j] = __float_as_uint(__fadd_rn(__uint_as_float(v[j]), __uint_as_float(more[j])));
            }
        }
    };
    const uint32_t toks = min(TT, P.tokens - m0);  // of this tile
    if (parts == 1) {
        if (warp < 4 && ok) {
#pragma unroll 1
            for (uint32_t c = 0; c < toks; c += 16) {
                uint32_t acc[16];
                float xs[16];  // before the stores, which the compiler must take for stores to xs, too
#pragma unroll
                for (uint32_t j = 0; j < 16; ++j) xs[j] = J.xs[m0 + min(c + j, toks - 1)];
                load_sums(c, acc);
                if (r < J.rows) {
#pragma unroll
                    for (uint32_t j = 0; j < 16; ++j)
                        if (c + j < toks) J.y[(size_t)(m0 + c + j) * J.rows + r] = scaled<DT>(acc[j], xs[j], ws);
                }
            }
        }
    } else {
        // every CTA of the cluster has finished with its stages: they now take the partial sums.
        // Token chunk c (of 4) is summed by CTA c % parts, from [c / parts][part][row][4 tokens].
        cluster_sync_all();
        if (warp < 4 && ok) {
#pragma unroll 1
            for (uint32_t c = 0; c < toks; c += 16) {
                uint32_t acc[16];
                load_sums(c, acc);
#pragma unroll
                for (uint32_t j = 0; j < 16; j += 4) {
                    if (c + j >= toks) break;
                    const uint32_t ch = (c + j) / 4, to = ch % parts, slot = ch / parts;
                    const uint32_t at = cluster_addr(base + ((slot * parts + rank) * kRowsTile + row) * 16, to);
                    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(acc[j]),
                                 "r"(acc[j + 1]), "r"(acc[j + 2]), "r"(acc[j + 3])
                                 : "memory");
                }
            }
        }
        cluster_sync_all();
        if (warp < 4 && r < J.rows) {
            for (uint32_t ch = rank, slot = 0; ch * 4 < toks; ch += parts, ++slot) {
                uint32_t sum[4] = {0, 0, 0, 0};
                float xs[4];
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) xs[j] = J.xs[m0 + min(ch * 4 + j, toks - 1)];
                for (uint32_t p = 0; p < parts; ++p) {
                    const uint32_t at = base + ((slot * parts + p) * kRowsTile + row) * 16;
                    uint32_t v[4];
                    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]),
                                 "=r"(v[3]) : "r"(at));
#pragma unroll
                    for (uint32_t j = 0; j < 4; ++j) {
                        if constexpr (DT == EQ_INT8)
                            sum[j] += v[j];
                        else
                            sum[j] = __float_as_uint(__fadd_rn(__uint_as_float(sum[j]), __uint_as_float(v[j])));
                    }
                }
#pragma unroll
                for (uint32_t j = 0; j < 4; ++j) {
                    if (ch * 4 + j < toks)
                        J.y[(size_t)(m0 + ch * 4 + j) * J.rows + r] = scaled<DT>(sum[j], xs[j], ws);
                }
            }
        }
    }
    if (J.n_out && warp < 4) {
        epilogue_sync<128>();  // this CTA's part of Y is written
        add_outliers<DT>(J, n0, m0, toks, rank, parts, tid, 128);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(P.tmem_cols) : "memory");
    }
}

// ---- pairs of SMs, persistent -------------------------------------------------------
// A cluster of two CTAs computes 256 weight rows x 256 tokens with
// cta_group::2 (M = 256): CTA q holds weight rows 128 q .. + 127 (half of A)
// and tokens 128 q .. + 127 (half of B) of each slab in its shared memory and
// the accumulator of its 128 rows for all 256 tokens in its tensor memory, twice
// (2 x 256 columns).
//   loader    (each CTA) after "empty" (CTA 0's commit, to both CTAs) its two
//             boxes, which complete on CTA 0's "full" barrier; CTA 0's loader
//             arms that barrier for the bytes of both
//   MMA lane  (CTA 0) per tile: waits until both CTAs' epilogues have read this
//             accumulator's previous tile ("free"), then per slab waits for
//             "full", issues 4 MMAs, commits to "empty" in both CTAs; at the
//             end commits to "done" of the accumulator in both
//   epilogue  (each CTA) 8 warps, a thread one row and half of the tokens: waits
//             for "done", takes the accumulator to registers (E4M3: adds it
//             to the parts of K before), arrives on CTA 0's "free"; behind the
//             last part scales and stores
constexpr uint32_t kPairTok = 256;
constexpr uint32_t kPairRows = 2 * kRowsTile;
constexpr uint32_t kPair8Stage = kWTile + 128 * kSlab;  // per CTA: 128 rows + 128 tokens of a slab
constexpr uint32_t kPair8Stages = 6;
constexpr size_t kPair8Smem = kPair8Stages * kPair8Stage + 1024;
static_assert(kPair8Smem <= 226u * 1024u, "shared memory per block");

template <int DT>
__device__ __forceinline__ void mma8_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t accumulate) {
    constexpr uint32_t idesc = instr_desc<DT>(kPairTok, kPairRows);
    if constexpr (DT == EQ_INT8)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
            "r"(accumulate)
            : "memory");
}

// A box into this CTA's shared memory that completes on a barrier of the pair's CTA 0.
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap *map, uint32_t x, uint32_t y,
                                            uint32_t cluster_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y),
        "r"(cluster_bar)
        : "memory");
}

// The parts of a tile's K that go through an accumulator of their own.
template <int DT>
__device__ __forceinline__ uint32_t segments(uint32_t slabs) {
    return DT == EQ_INT8 ? 1u : (slabs + kChain - 1) / kChain;
}

// Where a tile starts its walk through K (it wraps around): see the split kernel's loader.
__device__ __forceinline__ uint32_t first_slab(uint32_t local, uint32_t t_tiles, uint32_t slabs) {
    return (local % t_tiles * 3 + local / t_tiles * 7) % slabs;
}

// The epilogue of a cluster's tiles: one of eight warps, for the 32 accumulator lanes that it reaches (warp % 4) and
// half of the tokens.  False when a wait ran out here or elsewhere.  A warp that gives up still goes through its
// tiles, without waiting or storing: the eight meet at a barrier in every tile with super weights, however much
// later than the others one of them learns of it.
// The parts' sum stays in registers (128 of 168; a few loop values spill, 40 bytes).  Through Y (four warps, loads and stores of a part's outputs) 2048 tokens x 8192 x
// 28672 took 437 us in 3 parts and 680 in 14, here 417 to 435 in 14.
template <int DT>
__device__ __forceinline__ bool pair_epilogue(const A8Params &P, uint32_t cl, uint32_t n_clusters, uint32_t rank,
                                              uint32_t tmem, uint32_t done0, uint32_t free_c0,
                                              const volatile uint32_t *abort, uint32_t warp, uint32_t lane) {
    constexpr uint32_t kTok = kPairTok / 2;
    const uint32_t row = (warp & 3u) * 32u + lane, tok0 = (warp >> 2) * kTok;
    bool ok = true;
    uint32_t ti = 0;
    for (uint32_t tile = cl, jb = 0; tile < P.total_units; tile += n_clusters) {
        if (__any_sync(0xFFFFFFFFu, *abort != 0u)) ok = false;
        while (jb + 1 < P.n_jobs && tile >= P.jobs[jb + 1].first_unit) ++jb;
        const A8Job &J = P.jobs[jb];
        const uint32_t local = tile - J.first_unit;
        const uint32_t r = (local / P.t_tiles) * kPairRows + rank * kRowsTile + row;
        const uint32_t m0 = (local % P.t_tiles) * kPairTok;
        const float ws = r < J.rows ? J.ws[r] : 0.f;
        if (J.n_out && local == 0 && warp == 0 && rank == 0) check_outliers(J, lane, 32, P.status);
        const uint32_t segs = segments<DT>((J.cols + kSlab - 1) / kSlab);
        uint32_t sum[kTok];  // int32 or fp32 bits
#pragma unroll
        for (uint32_t j = 0; j < kTok; ++j) sum[j] = 0u;
#pragma unroll 1
        for (uint32_t seg = 0; seg < segs && ok; ++seg, ++ti) {
            const uint32_t a = ti & 1u;
            if (!warp_wait(done0 + 8 * a, (ti >> 1) & 1u)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t acc0 = tmem + (((warp & 3u) * 32u) << 16) + a * kPairTok + tok0;
#pragma unroll
            for (uint32_t c = 0; c < kTok; c += 16) {
                uint32_t acc[16];
                tmem_ld16(acc0 + c, acc);
#pragma unroll
                for (uint32_t j = 0; j < 16; ++j)
                    sum[c + j] = DT == EQ_INT8 ? acc[j]
                                               : __float_as_uint(__fadd_rn(__uint_as_float(sum[c + j]), __uint_as_float(acc[j])));
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(free_c0 + 8 * a);
        }
        if (ok) {
            const uint32_t t0 = m0 + tok0;
            float *y = J.y + (size_t)t0 * J.rows + r;
#pragma unroll
            for (uint32_t c = 0; c < kTok; c += 8) {
                float xs[8];  // before the stores, which the compiler must take for stores to xs, too
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j) xs[j] = J.xs[min(t0 + c + j, P.tokens - 1)];
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j, y += J.rows)
                    if (r < J.rows && t0 + c + j < P.tokens) *y = scaled<DT>(sum[c + j], xs[j], ws);
            }
        }
        if (J.n_out) {
            epilogue_sync<kPairEpilogue>();  // the tile's Y is written
            if (ok)
                add_outliers<DT>(J, r - row, m0, min(kPairTok, P.tokens - m0), 0, 1, warp * 32u + lane, kPairEpilogue);
        }
    }
    return ok;
}

template <int DT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    eq_gemm_a8_pair_kernel(const __grid_constant__ A8Params P) {
    constexpr uint32_t kStages = kPair8Stages;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) uint64_t full_s[kStages], empty_s[kStages], done_s[2], free_s[2];
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile uint32_t abort_s;
    const uint32_t tid = threadIdx.x, warp = warp_index(), lane = tid & 31u;
    const uint32_t rank = cluster_rank();
    const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t full0 = smem_u32(&full_s[0]), empty0 = smem_u32(&empty_s[0]);
    const uint32_t done0 = smem_u32(&done_s[0]), free0 = smem_u32(&free_s[0]);

    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&tmem_base_s)), "r"(2 * kPairTok) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (uint32_t st = 0; st < kStages; ++st) {
            mbar_init(full0 + 8 * st, 1);
            mbar_init(empty0 + 8 * st, 1);
        }
        for (uint32_t a = 0; a < 2; ++a) {
            mbar_init(done0 + 8 * a, 1);
            mbar_init(free0 + 8 * a, 16);  // (CTA 0) eight epilogue warps of each CTA
        }
        fence_mbar_init();
        abort_s = 0;
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    next_kernel_may_start();  // tensor memory is allocated
    previous_kernel_done();
    const uint32_t tmem = tmem_base_s;
    const uint32_t n_clusters = gridDim.x / 2, cl = blockIdx.x / 2;
    bool ok = true;

    if (warp == 8) {
        // ---- loader (both CTAs) ----
        const uint32_t full_c0 = cluster_addr(full0, 0);
        uint32_t st = 0, ph = 0, g = 0;
        for (uint32_t tile = cl, jb = 0; tile < P.total_units && ok; tile += n_clusters) {
            while (jb + 1 < P.n_jobs && tile >= P.jobs[jb + 1].first_unit) ++jb;
            const A8Job &J = P.jobs[jb];
            const uint32_t local = tile - J.first_unit;
            const uint32_t n0 = (local / P.t_tiles) * kPairRows + rank * kRowsTile;
            const uint32_t m0 = (local % P.t_tiles) * kPairTok + rank * 128u;
            const uint32_t slabs = (J.cols + kSlab - 1) / kSlab;
            uint32_t k = first_slab(local, P.t_tiles, slabs);
            for (uint32_t i = 0; i < slabs; ++i, ++g, k = k + 1 == slabs ? 0 : k + 1) {
                if (g >= kStages && !warp_wait(empty0 + 8 * st, ph ^ 1u)) {
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    const uint32_t buf = base + st * kPair8Stage;
                    if (rank == 0) mbar_expect_tx(full0 + 8 * st, 2 * kPair8Stage);
                    tma_2d_pair(buf, &J.tmap_w, k * kSlab, n0, full_c0 + 8 * st);
                    tma_2d_pair(buf + kWTile, &J.tmap_x, k * kSlab, m0, full_c0 + 8 * st);
                }
                __syncwarp();
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1u;
                }
            }
        }
        // the copies in flight land before the CTA leaves: both CTAs see it on the commits of the products
        // that read them ("empty"; what is left of the last round)
        for (uint32_t k = g > kStages ? g - kStages : 0; k < g; ++k)
            if (!warp_wait(empty0 + 8 * (k % kStages), (k / kStages) & 1u)) ok = false;
    } else if (warp == 9 && rank == 0) {
        // ---- MMA (CTA 0) ----
        const uint64_t a0 = slab_desc(base), b0 = slab_desc(base + kWTile);
        uint32_t st = 0, ph = 0, ti = 0;  // ti: accumulators filled so far
        for (uint32_t tile = cl, jb = 0; tile < P.total_units && ok; tile += n_clusters) {
            while (jb + 1 < P.n_jobs && tile >= P.jobs[jb + 1].first_unit) ++jb;
            const uint32_t slabs = (P.jobs[jb].cols + kSlab - 1) / kSlab, segs = segments<DT>(slabs);
            for (uint32_t seg = 0; seg < segs && ok; ++seg, ++ti) {
                const uint32_t a = ti & 1u, use = ti >> 1;  // accumulator, its use-th filling
                if (use > 0 && !warp_wait(free0 + 8 * a, (use - 1) & 1u)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t n = slabs / segs + (seg < slabs % segs);
                for (uint32_t k = 0; k < n; ++k) {
                    if (!warp_wait(full0 + 8 * st, ph)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t off = (uint64_t)((st * kPair8Stage) >> 4);
#pragma unroll
                        for (uint32_t kk = 0; kk < kSlab / kMmaK8; ++kk)
                            mma8_pair<DT>(tmem + a * kPairTok, a0 + off + 2u * kk, b0 + off + 2u * kk, k | kk);
                        tc_commit_pair(empty0 + 8 * st);
                        if (k + 1 == n) tc_commit_pair(done0 + 8 * a);
                    }
                    __syncwarp();
                    if (++st == kStages) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
            }
        }
        // no product may still run when the tensor memory is released
        if (ok)
            for (uint32_t k = ti > 2 ? ti - 2 : 0; k < ti; ++k)
                if (!warp_wait(done0 + 8 * (k & 1u), (k >> 1) & 1u)) ok = false;
    } else if (warp < 8) {
        // ---- epilogue (both CTAs) ----
        ok = pair_epilogue<DT>(P, cl, n_clusters, rank, tmem, done0, cluster_addr(free0, 0), &abort_s, warp, lane);
    }
    if (!ok) {
        abort_s = 1;
        atomicOr(P.status, EQ_DEV_TIMEOUT);
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync_all();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kPairTok) : "memory");
    }
}

// Failure-path check of the pair kernel's epilogue: its eight warps on one tile of a job with super weights, whose
// products are marked done.  Seven of them store the tile and wait at its barrier; the last first runs out a bounded
// wait on a barrier that nothing arrives on, raises the abort flag, and enters as a warp that has given up.  The
// block has to end, with EQ_DEV_TIMEOUT set and its tensor memory freed.
__global__ void __launch_bounds__(kPairEpilogue, 1) eq_a8_wait_timeout_kernel(const __grid_constant__ A8Params P) {
    __shared__ __align__(8) uint64_t never_s, done_s[2], free_s[2];
    __shared__ uint32_t tmem_base_s;
    __shared__ volatile uint32_t abort_s;
    const uint32_t tid = threadIdx.x, warp = warp_index(), lane = tid & 31u;
    const uint32_t never = smem_u32(&never_s), done0 = smem_u32(&done_s[0]), free0 = smem_u32(&free_s[0]);
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&tmem_base_s)), "r"(2 * kPairTok) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        mbar_init(never, 1);
        for (uint32_t a = 0; a < 2; ++a) {
            mbar_init(done0 + 8 * a, 1);
            mbar_init(free0 + 8 * a, 16);
        }
        fence_mbar_init();
        abort_s = 0;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base_s;
    const uint32_t zero[16] = {};
    for (uint32_t c = 0; c < kPairTok / 2; c += 16)
        tmem_st16(tmem + (((warp & 3u) * 32u) << 16) + (warp >> 2) * (kPairTok / 2) + c, zero);
    tmem_st_wait();
    tc_fence_before();
    __syncthreads();
    bool ok = true;
    if (warp == 0) warp_arrive(done0);
    if (warp == 7 && !warp_wait(never, 0u)) {
        ok = false;
        abort_s = 1;
        __syncwarp();
    }
    if (!pair_epilogue<EQ_INT8>(P, 0, 1, 0, tmem, done0, cluster_addr(free0, 0), &abort_s, warp, lane)) ok = false;
    if (!ok) atomicOr(P.status, EQ_DEV_TIMEOUT);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(2 * kPairTok) : "memory");
    }
}
__device__ uint32_t selftest_words[8];  // zeros: the job's scales, tokens, outputs and super weight

int encode_map8(CUtensorMap *map, const void *p, uint32_t rows, uint32_t cols, uint32_t box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return EQ_ERR_CUDA;
    const cuuint64_t dims[2] = {cols, rows};
    const cuuint64_t strides[1] = {cols};
    const cuuint32_t box[2] = {kSlab, box_rows};
    const cuuint32_t estr[2] = {1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? EQ_OK : EQ_ERR_CUDA;
}

int check_job(const eq_a8_job &j, uint32_t tokens) {
    if (j.dtype != EQ_INT8 && j.dtype != EQ_E4M3) return EQ_ERR_INVALID_ARG;
    if (!j.rows) return EQ_OK;
    if (j.rows > kMaxRows) return EQ_ERR_UNSUPPORTED;
    if (!j.cols || j.cols % 16 || j.cols > (j.dtype == EQ_INT8 ? kMaxInt8Cols : kMaxRows)) return EQ_ERR_UNSUPPORTED;
    if (!j.sym || !j.scale || (tokens && (!j.x8 || !j.x_scale || !j.y))) return EQ_ERR_INVALID_ARG;
    const auto at = [](const void *p) { return reinterpret_cast<uintptr_t>(p); };
    if (at(j.sym) % 16 || at(j.x8) % 16 || at(j.scale) % 4 || at(j.x_scale) % 4 || at(j.y) % 4)
        return EQ_ERR_INVALID_ARG;
    if (j.n_out && (!j.out_row || !j.out_col || !j.out_val || !j.out_stride || at(j.out_row) % 4 ||
                    at(j.out_col) % 4 || at(j.out_val) % 4))
        return EQ_ERR_INVALID_ARG;
    return EQ_OK;
}

// Launch shape.  Estimated SM clocks decide, from what one SM does: a split CTA's slab takes max(2 tok
// (products), bytes / 40 (copies)), a pair's 512 (both); memory delivers about 23 bytes per clock and SM
// when all run.  A round of CTAs costs about 4000 clocks besides (set-up, first copies, epilogue), sums
// that meet over the cluster 2000 more; the pairs' one round 8000 (a pair starts together, its last epilogue is
// 256 x 256).  8192 x 8192, us split and pairs, the estimate's choice in brackets:
//   tokens     32          65          128         256         512         1024
//   Int8   [16.5] 24.5 [17.9] 24.7 [21.4] 26.1  31.4 [27.0] 41.1 [33.9] 77.7 [59.3]
//   E4M3   [16.7] 25.1 [18.2] 25.5 [21.9] 27.1  32.9 [29.4] 46.0 [39.3] 85.0 [68.0]
// 131 x 4104 x 11008 Int8 [18.7] 35.1; 300 x 28672 x 8192 Int8 138 [96]; 256 x 8192 x 28672 E4M3 86 [88].
struct Shape {
    bool pair;
    uint32_t parts;  // CTAs that share a tile's K
};

// Accumulators of `tok` tokens that fit a CTA's share of the tensor memory: half of it while two CTAs of the split
// kernel fit an SM's shared memory (up to 64 tokens), so that neither waits for the other's.
uint32_t max_accs(uint32_t tok) { return (tok <= 64 ? 256 : 512) / tok; }

Shape pick_shape(const std::vector<const eq_a8_job *> &jobs, size_t at, size_t end, uint32_t tokens, uint32_t tok,
                 uint32_t sms, bool limited, bool chained) {
    if (limited) return {true, 1};
    const uint64_t t_tiles = (tokens + kSplitTok - 1) / kSplitTok, slots = tok <= 64 ? 2 * sms : sms;
    uint64_t units = 0, pair_units = 0, slabs = 0, min_slabs = ~0ull, bytes = 0;
    for (size_t k = at; k < end; ++k) {
        const eq_a8_job &q = *jobs[k];
        const uint64_t n = (q.cols + kSlab - 1) / kSlab;
        units += ((uint64_t)q.rows + kRowsTile - 1) / kRowsTile * t_tiles;
        pair_units += ((uint64_t)q.rows + kPairRows - 1) / kPairRows * t_tiles;
        slabs = std::max(slabs, n), min_slabs = std::min(min_slabs, n);
        bytes += (uint64_t)q.rows * q.cols + (uint64_t)tokens * q.cols + 4ull * tokens * q.rows;
    }
    const uint64_t memory = bytes / (23ull * sms);
    const auto rounds = [](uint64_t n, uint64_t of) { return (n + of - 1) / of; };
    Shape best{true, 1};
    uint64_t best_cost = ~0ull;
    // What an E4M3 part's accumulators reach.  Never more than 96 slabs: the estimate likes too few parts of a long K
    // (64 tokens x 8192 x 28672: 44 us in three, 50 in the two that it would take).
    const uint32_t reach = std::min(2 * kChain * max_accs(tok), 96u);
    const uint32_t least = chained ? (uint32_t)std::min<uint64_t>((slabs + reach - 1) / reach, kMaxSplit + 1) : 1;
    for (uint32_t parts = least; parts <= kMaxSplit && (parts == 1 || 2ull * parts <= min_slabs); ++parts) {
        const uint64_t slab = std::max<uint64_t>(2 * tok, (kWTile + (uint64_t)tok * kSlab) / 40);
        const uint64_t sm = rounds(units * parts, sms) * rounds(slabs, parts) * slab;
        const uint64_t cost = std::max(memory, sm) + rounds(units * parts, slots) * 4000 + (parts > 1 ? 2000 : 0);
        if (cost < best_cost) best = {false, parts}, best_cost = cost;
    }
    if (best_cost != ~0ull && sms >= 2 && std::max(memory, rounds(pair_units, sms / 2) * slabs * 512) + 8000 < best_cost) best = {true, 1};
    return best;
}

template <int DT>
int launch_type(const std::vector<const eq_a8_job *> &jobs, uint32_t tokens, uint32_t sms, bool limited,
                int32_t *d_status, cudaStream_t s) {
    for (size_t at = 0; at < jobs.size(); at += kMaxA8Jobs) {
        const size_t end = std::min(jobs.size(), at + kMaxA8Jobs);
        A8Params P{};
        P.status = d_status;
        P.tokens = tokens;
        // the split kernel's token tiles: as few as possible, of equal width
        P.t_tiles = (tokens + kSplitTok - 1) / kSplitTok;  // (the pair kernel's are 256 wide too)
        P.tok = ((tokens + P.t_tiles - 1) / P.t_tiles + 15) / 16 * 16;
        const Shape shape = pick_shape(jobs, at, end, tokens, P.tok, sms, limited, DT == EQ_E4M3);
        const bool pair = shape.pair;
        if (pair) P.tok = kPairTok;
        const uint32_t tile_rows = pair ? kPairRows : kRowsTile;
        uint64_t units = 0;
        for (size_t k = at; k < end; ++k) {
            const eq_a8_job &q = *jobs[k];
            A8Job &J = P.jobs[P.n_jobs++];
            if (const int rc = encode_map8(&J.tmap_w, q.sym, q.rows, q.cols, kRowsTile)) return rc;
            if (const int rc = encode_map8(&J.tmap_x, q.x8, tokens, q.cols, pair ? 128u : P.tok)) return rc;
            J.ws = q.scale, J.xs = q.x_scale, J.y = q.y, J.x8 = static_cast<const uint8_t *>(q.x8);
            J.out_row = q.out_row, J.out_col = q.out_col, J.out_val = q.out_val;
            J.n_out = q.n_out, J.out_stride = q.out_stride;
            J.rows = q.rows, J.cols = q.cols;
            J.first_unit = (uint32_t)units;
            units += (uint64_t)((q.rows + tile_rows - 1) / tile_rows) * P.t_tiles;
            if (units * kMaxSplit > 0x7FFFFFFFull) return EQ_ERR_UNSUPPORTED;
        }
        P.total_units = (uint32_t)units;
        const void *fn = (const void *)eq_gemm_a8_pair_kernel<DT>;
        size_t smem = kPair8Smem;
        uint32_t grid = 2 * (uint32_t)std::min<uint64_t>(units, sms / 2), parts = 1;
        if (!pair) {
            fn = (const void *)eq_gemm_a8_split_kernel<DT>;
            P.stage_bytes = kWTile + P.tok * kSlab;
            // two CTAs per SM up to 64 tokens: one's prologue and epilogue run under the other's loads
            const bool two = P.tok <= 64;
            smem = two ? kSplitSmem2 : kSplitSmem1;
            P.stages = std::min<uint32_t>(kMaxStages, (uint32_t)((smem - 1024) / P.stage_bytes));
            parts = shape.parts;
            P.accs = 1;
            if (DT == EQ_E4M3) {
                const uint32_t most = ((jobs[at]->cols + kSlab - 1) / kSlab + parts - 1) / parts;  // slabs; longest K first
                P.accs = std::min(max_accs(P.tok), (most + kChain - 1) / kChain);
            }
            for (P.tmem_cols = 32; P.tmem_cols < P.accs * P.tok;) P.tmem_cols *= 2;
            grid = (uint32_t)units * parts;
        }
        if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
            return EQ_ERR_CUDA;
        void *args[] = {&P};
        if (!launch_overlapped(fn, grid, pair ? kPairThreads : kA8Threads, smem, pair ? 0 : parts, args, s)) return EQ_ERR_CUDA;
    }
    return EQ_OK;
}

// Checks every job, then launches the Int8 ones and the E4M3 ones.
int a8_launch(const eq_a8_job *jobs, uint32_t n, uint32_t tokens, uint32_t sm_limit, int32_t *d_status,
              cudaStream_t s) try {
    if (!d_status || (n && !jobs)) return EQ_ERR_INVALID_ARG;
    if (tokens > kMaxRows) return EQ_ERR_UNSUPPORTED;
    for (uint32_t i = 0; i < n; ++i)
        if (const int rc = check_job(jobs[i], tokens)) return rc;
    std::vector<const eq_a8_job *> by_type[2];
    for (uint32_t i = 0; i < n; ++i)
        if (jobs[i].rows) by_type[jobs[i].dtype == EQ_E4M3].push_back(&jobs[i]);
    if (!tokens || (by_type[0].empty() && by_type[1].empty())) return EQ_OK;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
        return EQ_ERR_CUDA;
    const bool limited = sm_limit && sm_limit < (uint32_t)sms;
    if (limited) sms = (int)std::max(2u, sm_limit);
    for (auto &v : by_type)  // longest K first: the tile order ends with the short tiles
        std::stable_sort(v.begin(), v.end(), [](const eq_a8_job *a, const eq_a8_job *b) { return a->cols > b->cols; });
    if (const int rc = launch_type<EQ_INT8>(by_type[0], tokens, (uint32_t)sms, limited, d_status, s)) return rc;
    return launch_type<EQ_E4M3>(by_type[1], tokens, (uint32_t)sms, limited, d_status, s);
} catch (...) {  // host memory for the job lists
    return EQ_ERR_NOSPACE;
}

eq_a8_job model_job(const eq_model *m, uint32_t matrix, const void *sym, const void *x8, const float *xs, float *y) {
    const MatrixDesc &d = m->mats[matrix];
    eq_a8_job j{};
    j.sym = static_cast<const uint8_t *>(sym);
    j.scale = reinterpret_cast<const float *>(m->d_blob + d.scales_off);
    j.x8 = x8, j.x_scale = xs, j.y = y;
    j.rows = d.info.cols ? d.info.rows : 0;  // an empty matrix has no outputs
    j.cols = d.info.cols, j.dtype = d.info.dtype;
    j.n_out = d.info.n_outliers;
    if (j.n_out) {  // container records {row, col, value}
        j.out_row = reinterpret_cast<const uint32_t *>(m->d_blob + d.outliers_off);
        j.out_col = j.out_row + 1;
        j.out_val = reinterpret_cast<const float *>(j.out_row + 2);
        j.out_stride = 3;
    }
    return j;
}

}  // namespace

extern "C" EQW_API int eq_gemm_a8(const eq_a8_job *jobs, uint32_t n_jobs, uint32_t tokens, int32_t *d_status,
                                  cudaStream_t s) {
    const eqw::NvtxScope nvtx_range("eq_gemm_a8");
    return a8_launch(jobs, n_jobs, tokens, 0, d_status, s);
}

extern "C" EQW_API int eq_gemm_symbols_a8(const eq_model *m, uint32_t matrix, const void *d_sym, const void *d_x8,
                                          const float *d_x_scale, uint32_t tokens, float *d_y, int32_t *d_status,
                                          cudaStream_t s) {
    const eqw::NvtxScope nvtx_range("eq_gemm_symbols_a8");
    if (!m || matrix >= m->mats.size()) return EQ_ERR_INVALID_ARG;
    const eq_a8_job j = model_job(m, matrix, d_sym, d_x8, d_x_scale, d_y);
    return a8_launch(&j, 1, tokens, m->sm_limit, d_status, s);
}

extern "C" EQW_API int eq_gemm_symbols_a8_block(const eq_model *m, uint32_t layer, const void *const *d_syms,
                                                const void *const *d_x8s, const float *const *d_x_scales,
                                                uint32_t tokens, float *const *d_ys, uint32_t count,
                                                int32_t *d_status, cudaStream_t s) try {
    const eqw::NvtxScope nvtx_range("eq_gemm_symbols_a8_block");
    if (!m || layer >= m->n_layers) return EQ_ERR_INVALID_ARG;
    const uint32_t first = m->layer_first[layer], n = m->layer_count[layer];
    if (count != n || (n && (!d_syms || !d_x8s || !d_x_scales || !d_ys))) return EQ_ERR_INVALID_ARG;
    std::vector<eq_a8_job> jobs(n);
    for (uint32_t i = 0; i < n; ++i) jobs[i] = model_job(m, first + i, d_syms[i], d_x8s[i], d_x_scales[i], d_ys[i]);
    return a8_launch(jobs.data(), n, tokens, m->sm_limit, d_status, s);
} catch (...) {
    return EQ_ERR_NOSPACE;
}

extern "C" EQW_API int eq_selftest_a8_wait_timeout(int32_t *d_status, cudaStream_t s) {
    if (!d_status) return EQ_ERR_INVALID_ARG;
    void *words = nullptr;
    if (cudaGetSymbolAddress(&words, selftest_words) != cudaSuccess) return EQ_ERR_CUDA;
    A8Params P{};
    P.status = d_status;
    P.tokens = P.t_tiles = P.n_jobs = P.total_units = 1;
    A8Job &J = P.jobs[0];  // 1 x 16, one token, one super weight: all zero
    J.ws = J.xs = J.out_val = static_cast<const float *>(words);
    J.out_row = J.out_col = static_cast<const uint32_t *>(words);
    J.x8 = static_cast<const uint8_t *>(words);
    J.y = static_cast<float *>(words) + 7;
    J.rows = J.n_out = J.out_stride = 1, J.cols = 16;
    eq_a8_wait_timeout_kernel<<<1, kPairEpilogue, 0, s>>>(P);
    return cudaGetLastError() == cudaSuccess ? EQ_OK : EQ_ERR_CUDA;
}
