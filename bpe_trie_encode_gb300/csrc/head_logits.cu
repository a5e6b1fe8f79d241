// head_logits.cu -- 8-bit matrix product with a scale per block of 128.
//
//   out[r, t] = sum_b xs[r, b] ws[t / 128, b] (sum_{k in b} x8[r, k] w8[t, k])
//
// The inner sums run on the tensor cores (tcgen05, e4m3 x e4m3, 32-bit
// accumulators in tensor memory), one block of 128 columns at a time; because
// every block has scales of its own, each block's 32-bit sums are read back
// and added, times their scales, to accumulators that stay in registers.  TMA
// fills a ring of shared-memory stages, one thread issues the products, the
// other warps scale and add; tensor memory holds several blocks' sums, so that
// the products of the next blocks run meanwhile.
#include "head.cuh"

#include <cudaTypedefs.h>

#include <type_traits>

#include "device.cuh"
#include "internal.h"
#include "tc.cuh"

namespace bpe {
namespace {

constexpr int kBlock = (int)BPE_HEAD_BLOCK;   // columns per scale = bytes per stage row

struct LogitsParams {
    const float *xs, *ws;
    void *out;
    uint64_t xs_row, xs_blk, ws_row, ws_blk, out_stride;
    uint32_t n_rows, n_tok, blocks;
    bool tma_out;                // the output's rows start on 16 bytes
    uint32_t *status;
    long long stall;             // BPE_OPT_TEST_STALL_HEAD
};

// ------------------------------------------------------------- few rows ----
// Up to 64 rows: the bound is reading the weights once.  The weights are the
// product's 128-row side, the kN rows of x the other.  Each SM streams its own
// contiguous share of the vocabulary, in steps of 16 tokens, through one
// CTA's ring of stages: shares are equal to within a step, so that all SMs end
// together, and a vocabulary of a few thousand tokens still spreads over all of
// them.  A lane of tensor memory is a token; row r's scale comes from lane r by
// a shuffle, the token's own is the lane's.  A stage has its own columns of
// tensor memory, and is loaded again when its sums have been read: the warp
// that multiplies, whose loop of about 300 cycles a block must stay below the
// 700 that 16 KB take to arrive, waits on one barrier and signals one (with two
// of each, 520 cycles, it was the bound).  Measured: 1 x 65,536 x 8,192 in 87 us,
// 6.1 TB/s; 1 x 32,256 x 4,096 in 25 to 26 us, 5.1 TB/s with the launch; 64 x
// 65,536 x 4,096 in 57 us, 5.0 TB/s.  That last one is not short of loads on the
// way (128-row tiles, below, have 96 KB of weights under way on an SM, not 128,
// and took 53): its adding warps take 8 instructions a sum, a shuffle and a
// product of scales among them, and 60% of the issue slots; a stage takes nine
// loads where a 128-row tile's takes two.
constexpr int kStep = 16;          // tokens per load

template <int kN> struct Few {
    static constexpr int kGroups = kN == 16 ? 2 : 4;            // of 4 warps that scale and add, each a part of the rows
    static constexpr int kThreads = kGroups * 128 + 64;         // and 1 warp loads, 1 multiplies
    static constexpr int kStage = (128 + kN) * kBlock;
    static constexpr int kStages = kN == 16 ? 12 : kN == 32 ? 11 : 8;
    static constexpr int kCols = kN * kStages <= 256 ? 256 : 512;   // of tensor memory, kN for each stage
    static_assert(kN * kStages <= kCols, "tensor memory");
    static constexpr int kSmem = kStages * kStage + 1024 + 512;
    static_assert(kSmem <= 232448, "shared memory of a CTA");
};

template <int kN, typename O>
__global__ void __launch_bounds__(Few<kN>::kThreads, 1)
k_logits_few(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, LogitsParams P,
             uint32_t share) {
    using F = Few<kN>;
    constexpr int kStages = F::kStages, kLoader = F::kGroups * 4;
    constexpr int kPart = kN / F::kGroups;   // rows that a warp adds
    extern __shared__ uint8_t raw[];
    uint8_t *base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    const uint32_t tiles = smem_u32(base);
    const uint32_t bars = tiles + kStages * F::kStage;
    uint32_t *extra = (uint32_t *)(base + kStages * F::kStage + 448);   // [0] tensor memory, [1] gave up
    auto full = [&](int s) { return bars + 8 * s; };
    auto done = [&](int s) { return bars + 8 * (kStages + s); };
    auto taken = [&](int s) { return bars + 8 * (2 * kStages + s); };
    const int warp = __shfl_sync(kFull, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t begin = min(P.n_tok, blockIdx.x * share), end = min(P.n_tok, begin + share);
    volatile uint32_t *gave_up = extra + 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) mbar_init(full(s), 1), mbar_init(done(s), 1), mbar_init(taken(s), kLoader);
        extra[1] = 0;
        mbar_init_fence();
    }
    if (warp == kLoader + 1) tmem_alloc(smem_u32(extra), F::kCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = extra[0];

    if (warp == kLoader) {
        tma_prefetch_map(&map_w);
        tma_prefetch_map(&map_x);
        int s = 0;
        uint32_t phase = 1, issued = 0;
        for (uint32_t tok = P.stall == blockIdx.x ? end : begin; tok < end && !__any_sync(kFull, *gave_up); tok += 128) {
            const uint32_t steps = (min(128u, end - tok) + kStep - 1) / kStep;
            for (uint32_t b = 0; b < P.blocks; b++) {
                if (!__all_sync(kFull, mbar_wait(taken(s), phase))) { *gave_up = 1; break; }
                if (elect_one()) {
                    const uint32_t at = tiles + s * F::kStage;
                    mbar_expect(full(s), (steps * kStep + kN) * kBlock);
                    const int x = (int)(b * kBlock);
                    tma_load(at + 128 * kBlock, &map_x, x, 0, full(s));
                    for (uint32_t i = 0; i < steps; i++)   // what a short tile leaves of the stage keeps old weights, whose sums go nowhere
                        tma_load(at + i * kStep * kBlock, &map_w, x, (int)(tok + i * kStep), full(s));
                }
                issued++;
                if (++s == kStages) s = 0, phase ^= 1;
            }
        }
        if (*gave_up)   // no copy may be in flight when the CTA ends
            for (uint32_t i = issued > kStages ? issued - kStages : 0; i < issued; i++)
                mbar_wait(full(i % kStages), (i / kStages) & 1);
    } else if (warp == kLoader + 1) {
        int s = 0;
        uint32_t phase = 0;
        const uint32_t w0 = operand_lo(tiles), x0 = operand_lo(tiles + 128 * kBlock);
        for (uint32_t tok = begin; tok < end && !__any_sync(kFull, *gave_up); tok += 128) {
            for (uint32_t b = 0; b < P.blocks; b++) {
                if (!__all_sync(kFull, mbar_wait(full(s), phase))) { *gave_up = 1; break; }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t w = w0 + s * (F::kStage >> 4), x = x0 + s * (F::kStage >> 4), d = tmem + s * kN;
                    constexpr uint32_t kInstr = e4m3_instr(128, kN);
                    mma_e4m3<false>(d, w, x, kInstr);
                    mma_e4m3<true>(d, w + 2, x + 2, kInstr);
                    mma_e4m3<true>(d, w + 4, x + 4, kInstr);
                    mma_e4m3<true>(d, w + 6, x + 6, kInstr);
                    mma_commit(done(s));
                }
                if (++s == kStages) s = 0, phase ^= 1;
            }
        }
    } else {
        constexpr int kPer = (kPart + 31) / 32;   // row scales that a lane holds
        const int quarter = warp & 3, col0 = (warp >> 2) * kPart;
        const uint32_t last = P.blocks - 1;
        int s = 0;
        uint32_t phase = 0;
        struct Scales { float w, x[kPer]; };
        const float *xs[kPer];
#pragma unroll
        for (int i = 0; i < kPer; i++)   // lanes past the rows read a scale that nothing uses
            xs[i] = P.xs + min((uint32_t)(col0 + i * 32 + lane), P.n_rows - 1) * P.xs_row;
        const uint32_t mine = tmem + ((uint32_t)quarter << 21) + col0;
        bool ok = true;   // once a wait has given up: NaN for what is left
        for (uint32_t tok = begin; tok < end; tok += 128) {
            const uint32_t t = tok + quarter * 32 + lane;
            const float *ws = P.ws + (uint64_t)(min(t, P.n_tok - 1) / kBlock) * P.ws_row;
            auto load = [&](uint32_t b) {
                Scales v;
                b = min(b, last);
                v.w = ws[b * P.ws_blk];
#pragma unroll
                for (int i = 0; i < kPer; i++) v.x[i] = xs[i][b * P.xs_blk];
                return v;
            };
            float acc[kPart];
#pragma unroll
            for (int c = 0; c < kPart; c++) acc[c] = 0.0f;
            auto add = [&](const float (&d)[kPart], const Scales &by) {
#pragma unroll
                for (int c = 0; c < kPart; c++)
                    acc[c] = fmaf(d[c], by.w * __shfl_sync(kFull, by.x[c / 32], c), acc[c]);
            };
            // two blocks at a time: half the waits, and a block's scales have two blocks' time to arrive
            Scales a = load(0), b2 = load(1);
            for (uint32_t b = 0; b < P.blocks && ok; b += 2) {
                const bool two = b + 1 < P.blocks;
                const int s1 = s + 1 == kStages ? 0 : s + 1;
                const uint32_t phase1 = s1 ? phase : phase ^ 1;
                const bool second = two && lane >= 16;   // half of the lanes watch each barrier
                if (!__all_sync(kFull, mbar_wait(second ? done(s1) : done(s), second ? phase1 : phase))) { ok = false, *gave_up = 1; break; }
                tc_fence_after();
                float d[kPart], d1[kPart];
                tmem_load(d, mine + s * kN);
                tmem_load(d1, mine + (two ? s1 : s) * kN);
                tmem_wait(d);
                tmem_wait(d1);
                tc_fence_before();
                if (lane == 0) {
                    mbar_arrive(taken(s));
                    if (two) mbar_arrive(taken(s1));
                }
                add(d, a);
                a = load(b + 2);
                if (two) add(d1, b2);
                b2 = load(b + 3);
                s = s1, phase = phase1;
                if (two && ++s == kStages) s = 0, phase ^= 1;
            }
            if (!ok) {
#pragma unroll
                for (int c = 0; c < kPart; c++) acc[c] = NAN;
            }
            if (t < end) {
                O *out = (O *)P.out + t;
#pragma unroll
                for (int c = 0; c < kPart; c++)
                    if (col0 + c < P.n_rows) out[(uint64_t)(col0 + c) * P.out_stride] = from_f32<O>(acc[c]);
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kLoader + 1) tmem_free(tmem, F::kCols);
    if (threadIdx.x == 0 && *gave_up) *P.status = DERR_TIMEOUT;
}

// ------------------------------------------------------------ many rows ----
// The rows of x are the product's row side, 256 tokens the other.  A tile is
// 128 rows by one CTA, or 256 by a pair of CTAs that share the tokens' side (a
// pair reads a third less from L2 than two CTAs would).  Persistent CTAs take
// tiles in turn, rows fastest, so that those that run together read the same
// weights from L2.  Two sets of sums fill the 512 columns of tensor memory.  A
// thread that adds holds one row and 64 tokens, which are of one weight scale:
// its factor is one number per block.  16 such warps, 4 per scheduler, cover
// the latency of reading tensor memory.  The tile leaves through shared memory
// by TMA while the next one is under way.  Measured: 4,096 x 32,256 x 4,096 in
// 374 us (2.9 PFLOP/s) after a pause, 417 us when run on end; a block takes 800
// cycles of a CTA's tensor core where products alone, without scales, took
// 750; the rest is 2,000 cycles at each tile's end.  333 x 250,000 x 1,040, 9
// blocks a tile, 135 us: those ends are a fifth of it, waits for weights have
// not been measured apart.
constexpr int kManyThreads = 576;   // 16 warps scale and add, 1 loads, 1 multiplies
constexpr int kManyToks = 256;
constexpr int kOutBytes = 128 * 128;   // of one group of 4 warps: 128 rows of 128 bytes

template <int kCtas> struct Many {
    static constexpr int kRows = 128 * kCtas;
    static constexpr int kStages = kCtas == 1 ? 3 : 5;
    static constexpr int kToks = kManyToks / kCtas;                 // weights that a CTA loads
    static constexpr int kStage = (128 + kToks) * kBlock;
    static constexpr int kSmem = kStages * kStage + 4 * kOutBytes + 1024 + 256;
    static_assert(kSmem <= 232448, "shared memory of a CTA");
};

// A row's part of a tile, up to 128 bytes in swizzled shared memory, to a place that TMA cannot write: lane j of 8 writes
// the j-th 16 bytes that are aligned in the output, and element j of what is left before and after them.  Stores of one
// element a lane took 438 us
// against 410 for 779 x 142,605 x 2,896, and 134 against 108 for 1,547 x 53,514 x 433.
template <typename O>
__device__ __forceinline__ void store_part(O *to, const uint8_t *row, uint32_t swizzle, uint32_t n, uint32_t j) {
    constexpr uint32_t kSize = sizeof(O), kVec = 16 / kSize;
    auto chunk = [&](uint32_t c) { return *reinterpret_cast<const uint4 *>(row + ((c ^ swizzle) << 4)); };
    auto one = [&](uint32_t i) { to[i] = *reinterpret_cast<const O *>(row + (((i / kVec) ^ swizzle) << 4) + i % kVec * kSize); };
    const uint32_t before = (16 - ((uint32_t)(uintptr_t)to & 15)) & 15, skip = before / kSize;
    if ((j + 1) * kVec + skip <= n) {
        uint4 v = chunk(j);
        if (before) {
            const uint4 h = chunk(j + 1);   // within the 128 bytes: skip > 0 elements of it are still of the n
            if (before & 8) v.x = v.z, v.y = v.w, v.z = h.x, v.w = h.y;
            uint32_t e = before & 8 ? h.z : h.x, f = before & 8 ? h.w : h.y;
            if (before & 4) v.x = v.y, v.y = v.z, v.z = v.w, v.w = e, e = f;
            if (kSize == 2 && (before & 2))
                v.x = __funnelshift_r(v.x, v.y, 16), v.y = __funnelshift_r(v.y, v.z, 16), v.z = __funnelshift_r(v.z, v.w, 16),
                v.w = __funnelshift_r(v.w, e, 16);
        }
        *reinterpret_cast<uint4 *>(to + skip + j * kVec) = v;
    }
    if (j < min(skip, n)) one(j);
    if (n > skip) {
        const uint32_t rest = (n - skip) % kVec;
        if (j < rest) one(n - rest + j);
    }
}

// A barrier of a group's four warps: whether all of them have their sums.  They leave a tile, and the loop, together:
// a warp whose wait gave up by itself would be missed at the barriers that follow, which have no limit.
__device__ __forceinline__ bool group_all(uint32_t bar, bool ok) {
    uint32_t all;
    asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %2, 0;\nbar.red.and.pred q, %1, 128, p;\nselp.u32 %0, 1, 0, q;\n}"
                 : "=r"(all) : "r"(bar), "r"((uint32_t)ok) : "memory");
    return all != 0;
}

template <typename O, int kCtas>
__global__ void __launch_bounds__(kManyThreads, 1)
k_logits_many(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
              const __grid_constant__ CUtensorMap map_out, LogitsParams P) {
    using M = Many<kCtas>;
    constexpr int kStages = M::kStages;
    extern __shared__ uint8_t raw[];
    uint8_t *base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    const uint32_t tiles = smem_u32(base);
    uint8_t *outs = base + kStages * M::kStage;
    uint8_t *after = outs + 4 * kOutBytes;
    const uint32_t bars = smem_u32(after);
    uint32_t *extra = (uint32_t *)(after + 128);   // [0] tensor memory, [1] gave up
    auto full = [&](int s) { return bars + 8 * s; };               // a pair's: rank 0's
    auto empty = [&](int s) { return bars + 8 * (kStages + s); };
    auto done = [&](int b) { return bars + 8 * (2 * kStages + b); };
    auto taken = [&](int b) { return bars + 8 * (2 * kStages + 2 + b); };   // a pair's: rank 0's
    const int warp = __shfl_sync(kFull, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x % kCtas, team = blockIdx.x / kCtas, teams = gridDim.x / kCtas;
    const uint32_t row_tiles = (P.n_rows + M::kRows - 1) / M::kRows, tok_tiles = (P.n_tok + kManyToks - 1) / kManyToks;
    const uint32_t n_tiles = row_tiles * tok_tiles;
    volatile uint32_t *gave_up = extra + 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; s++) mbar_init(full(s), 1), mbar_init(empty(s), 1);
        for (int b = 0; b < 2; b++) mbar_init(done(b), 1), mbar_init(taken(b), 16 * kCtas);
        extra[1] = 0;
        mbar_init_fence();
    }
    if (warp == 17) {
        if (kCtas == 1)
            tmem_alloc(smem_u32(extra), 512);
        else
            tmem_alloc_pair(smem_u32(extra), 512);
    }
    tc_fence_before();
    if (kCtas == 1)
        __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    tc_fence_after();
    const uint32_t tmem = extra[0];

    if (warp == 16) {
        tma_prefetch_map(&map_w);
        tma_prefetch_map(&map_x);
        int s = 0;
        uint32_t phase = 1, issued = 0;
        for (uint32_t i = P.stall == blockIdx.x ? n_tiles : team; i < n_tiles && !__any_sync(kFull, *gave_up); i += teams) {
            const int row0 = (int)(i % row_tiles * M::kRows + rank * 128);
            const int tok0 = (int)(i / row_tiles * kManyToks + rank * M::kToks);
            for (uint32_t b = 0; b < P.blocks; b++) {
                if (!__all_sync(kFull, mbar_wait(empty(s), phase))) { *gave_up = 1; break; }
                const uint32_t at = tiles + s * M::kStage;
                if (elect_one()) {
                    if (rank == 0) mbar_expect(full(s), M::kStage * kCtas);
                    if (kCtas == 1) {
                        tma_load(at, &map_x, (int)(b * kBlock), row0, full(s));
                        tma_load(at + 128 * kBlock, &map_w, (int)(b * kBlock), tok0, full(s));
                    } else {
                        tma_load_pair(at, &map_x, (int)(b * kBlock), row0, full(s));
                        tma_load_pair(at + 128 * kBlock, &map_w, (int)(b * kBlock), tok0, full(s));
                    }
                }
                issued++;
                if (++s == kStages) s = 0, phase ^= 1;
            }
        }
        if (*gave_up && rank == 0)   // no copy may be in flight when the CTA ends
            for (uint32_t i = issued > kStages ? issued - kStages : 0; i < issued; i++)
                mbar_wait(full(i % kStages), (i / kStages) & 1);
    } else if (warp == 17) {
        if (rank == 0) {
            int s = 0, buf = 0;
            uint32_t phase = 0, bphase = 1;
            const uint32_t x0 = operand_lo(tiles), w0 = operand_lo(tiles + 128 * kBlock);
            for (uint32_t i = team; i < n_tiles && !__any_sync(kFull, *gave_up); i += teams) {
                for (uint32_t b = 0; b < P.blocks; b++) {
                    if (!__all_sync(kFull, mbar_wait(taken(buf), bphase) && mbar_wait(full(s), phase))) { *gave_up = 1; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t x = x0 + s * (M::kStage >> 4), w = w0 + s * (M::kStage >> 4), d = tmem + buf * kManyToks;
                        constexpr uint32_t kInstr = e4m3_instr(M::kRows, kManyToks);
                        if (kCtas == 1) {
                            mma_e4m3<false>(d, x, w, kInstr);
                            mma_e4m3<true>(d, x + 2, w + 2, kInstr);
                            mma_e4m3<true>(d, x + 4, w + 4, kInstr);
                            mma_e4m3<true>(d, x + 6, w + 6, kInstr);
                            mma_commit(done(buf));
                            mma_commit(empty(s));
                        } else {
                            mma_e4m3_pair<false>(d, x, w, kInstr);
                            mma_e4m3_pair<true>(d, x + 2, w + 2, kInstr);
                            mma_e4m3_pair<true>(d, x + 4, w + 4, kInstr);
                            mma_e4m3_pair<true>(d, x + 6, w + 6, kInstr);
                            mma_commit_pair(done(buf));
                            mma_commit_pair(empty(s));
                        }
                    }
                    if (++s == kStages) s = 0, phase ^= 1;
                    if (++buf == 2) buf = 0, bphase ^= 1;
                }
            }
        }
    } else {
        const int quarter = warp & 3, group = warp >> 2;
        uint8_t *mine = outs + group * kOutBytes;   // the group's 128 rows of 128 bytes, swizzled as TMA reads them
        const uint32_t r = quarter * 32 + lane;
        constexpr int kPer = 128 / sizeof(O);       // tokens in 128 bytes
        constexpr int kVec = 16 / sizeof(O);
        int buf = 0;
        uint32_t bphase = 0;
        const uint32_t last = P.blocks - 1;
        // the team's next tile is row_step tiles of rows and tok_step of tokens further
        const uint32_t row_step = teams % row_tiles, tok_step = teams / row_tiles;
        uint32_t row_tile = team % row_tiles, tok_tile = team / row_tiles;
        const float *xs, *ws;
        float sx0, sw0, sx1, sw1;   // the scales of a tile's first two blocks
        auto begin = [&] {
            xs = P.xs + (uint64_t)min(row_tile * M::kRows + rank * 128 + r, P.n_rows - 1) * P.xs_row;
            ws = P.ws + (uint64_t)min((tok_tile * kManyToks + group * 64) / kBlock, (P.n_tok - 1) / kBlock) * P.ws_row;
            sx0 = xs[0], sw0 = ws[0], sx1 = xs[min(1u, last) * P.xs_blk], sw1 = ws[min(1u, last) * P.ws_blk];
        };
        auto advance = [&] {
            row_tile += row_step, tok_tile += tok_step;
            if (row_tile >= row_tiles) row_tile -= row_tiles, tok_tile++;
        };
        if (tok_tile < tok_tiles) begin();
        while (tok_tile < tok_tiles) {
            float acc[64];
            bool ok = true;
            const float *const tx = xs, *const tw = ws;
            float ax = sx0, aw = sw0, bx = sx1, bw = sw1;
            auto add = [&](uint32_t b, auto first) {
                const float s = ax * aw;
                ax = bx, aw = bw;
                bx = tx[min(b + 2, last) * P.xs_blk];
                bw = tw[min(b + 2, last) * P.ws_blk];
                if (!__all_sync(kFull, mbar_wait(done(buf), bphase))) { ok = false; return; }
                tc_fence_after();
                const uint32_t at = tmem + ((uint32_t)quarter << 21) + buf * kManyToks + group * 64;
#pragma unroll
                for (int c0 = 0; c0 < 64; c0 += 16) {   // 16 at a time: 96 registers is what 18 warps have
                    float d[16];
                    tmem_load(d, at + c0);
                    tmem_wait(d);
                    if (c0 == 48) {
                        tc_fence_before();
                        if (lane == 0) {
                            if (kCtas == 1)
                                mbar_arrive(taken(buf));
                            else
                                mbar_arrive_far(taken(buf), 0);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 16; c++) acc[c0 + c] = decltype(first)::value ? d[c] * s : fmaf(d[c], s, acc[c0 + c]);
                }
                if (++buf == 2) buf = 0, bphase ^= 1;
            };
            add(0, std::true_type());
            for (uint32_t b = 1; b < P.blocks && ok; b++) add(b, std::false_type());
            const uint32_t row0 = row_tile * M::kRows + rank * 128, tok0 = tok_tile * kManyToks + group * 64;
            if (P.tma_out && quarter == 0 && lane == 0) tma_store_wait();
            if (!group_all(1 + group, ok)) { *gave_up = 1; break; }
            advance();
            if (tok_tile < tok_tiles) begin();   // the next tile's first scales arrive while this one leaves
#pragma unroll
            for (int c0 = 0; c0 < 64; c0 += kPer) {
                // TMA ends a row at a whole 16 bytes: a last part that does not is stored by threads
                const uint32_t t = tok0 + c0;
                const bool by_tma = P.tma_out && (t + kPer <= P.n_tok || P.n_tok % kVec == 0);
                if (c0 > 0) {
                    if (P.tma_out && quarter == 0 && lane == 0) tma_store_wait();
                    asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
                }
#pragma unroll
                for (int j = 0; j < 8; j++)
                    *reinterpret_cast<uint4 *>(mine + r * 128 + ((j ^ (r & 7)) << 4)) = pack16(acc + c0 + j * kVec, O());
                if (by_tma) fence_for_tma();
                asm volatile("bar.sync %0, 128;" ::"r"(1 + group) : "memory");
                if (by_tma) {
                    if (quarter == 0 && lane == 0 && row0 < P.n_rows && t < P.n_tok)
                        tma_store(&map_out, (int)t, (int)row0, smem_u32(mine));
                } else {
                    for (uint32_t q = (threadIdx.x & 127) / 8; q < 128 && row0 + q < P.n_rows; q += 16)
                        if (t < P.n_tok)
                            store_part((O *)P.out + (row0 + q) * P.out_stride + t, mine + q * 128, q & 7,
                                       min((uint32_t)kPer, P.n_tok - t), threadIdx.x & 7);
                }
            }
        }
        if (P.tma_out && quarter == 0 && lane == 0) tma_store_wait();
        for (; tok_tile < tok_tiles; advance()) {   // a wait gave up: NaN for what is left
            const uint32_t row = row_tile * M::kRows + rank * 128 + r, tok0 = tok_tile * kManyToks + group * 64;
            if (row < P.n_rows)
                for (uint32_t t = tok0; t < tok0 + 64 && t < P.n_tok; t++)
                    ((O *)P.out)[row * P.out_stride + t] = from_f32<O>(NAN);
        }
    }
    __syncwarp();
    tc_fence_before();
    if (kCtas == 1)
        __syncthreads();
    else
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    tc_fence_after();
    if (warp == 17) {
        if (kCtas == 1)
            tmem_free(tmem, 512);
        else
            tmem_free_pair(tmem, 512);
    }
    if (threadIdx.x == 0 && *gave_up) *P.status = DERR_TIMEOUT;
}

// -------------------------------------------------------------- the host ---
// Rows that do not start on 16 bytes, copied to rows that do: 16 bytes a thread, from the five aligned words that hold
// them.  A word is read only if a byte of the row lies in it.
__global__ void __launch_bounds__(256) k_head_align(const uint8_t *__restrict__ src, uint64_t stride, uint32_t rows,
                                                    uint32_t dim, uint8_t *__restrict__ dst, uint32_t dst_stride) {
    const uint32_t each = dst_stride / 16;
    const uint64_t parts = (uint64_t)rows * each;
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < parts; i += gridDim.x * 256ull) {
        const uint64_t r = i / each;
        const uint32_t c = (uint32_t)(i % each) * 16;
        const uintptr_t from = (uintptr_t)(src + r * stride + c), end = (uintptr_t)(src + r * stride + dim);
        const uint32_t *word = (const uint32_t *)(from & ~(uintptr_t)3);
        const uint32_t shift = (uint32_t)(from & 3) * 8;
        uint32_t w[5], v[4];
#pragma unroll
        for (int j = 0; j < 5; j++) w[j] = (uintptr_t)(word + j) < end ? __ldg(word + j) : 0;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            v[j] = __funnelshift_r(w[j], w[j + 1], shift);
            const int left = (int)dim - (int)(c + 4 * j);   // bytes of the row from here on
            if (left < 4) v[j] = left <= 0 ? 0 : v[j] & ((1u << 8 * left) - 1);
        }
        *(uint4 *)(dst + r * dst_stride + c) = make_uint4(v[0], v[1], v[2], v[3]);
    }
}

typedef PFN_cuTensorMapEncodeTiled_v12000 EncodeFn;

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return (EncodeFn) nullptr;
        }
        return (EncodeFn)p;
    }();
    return fn;
}

// The tile map of an 8-bit matrix, box_rows x 128 columns; columns past dim read as 0.  A load ends a row at the byte
// (rows padded with NaN to 16 bytes give the same bits), where a store ends it at whole 16 bytes.
int encode_map(bpe_ctx *ctx, CUtensorMap *map, const uint8_t *p, uint64_t stride, uint32_t rows, uint32_t dim, uint32_t box_rows) {
    EncodeFn fn = encode_fn();
    if (!fn) return fail(ctx, BPE_ERR_CUDA, "head_logits: the driver has no cuTensorMapEncodeTiled");
    const cuuint64_t size[2] = {dim, rows}, strides[1] = {stride};
    const cuuint32_t box[2] = {(cuuint32_t)kBlock, box_rows}, step[2] = {1, 1};
    const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, (void *)p, size, strides, box, step,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(ctx, BPE_ERR_CUDA, "head_logits: cuTensorMapEncodeTiled returned %d", (int)r);
    return BPE_OK;
}

// The output's map, for tiles of 128 rows and 128 bytes.
template <typename O>
int encode_out(bpe_ctx *ctx, CUtensorMap *map, const LogitsParams &P) {
    EncodeFn fn = encode_fn();
    if (!fn) return fail(ctx, BPE_ERR_CUDA, "head_logits: the driver has no cuTensorMapEncodeTiled");
    const CUtensorMapDataType type = sizeof(O) == 4 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_UINT16;
    const cuuint64_t size[2] = {P.n_tok, P.n_rows}, strides[1] = {P.out_stride * sizeof(O)};
    const cuuint32_t box[2] = {(cuuint32_t)(128 / sizeof(O)), 128}, step[2] = {1, 1};
    const CUresult r = fn(map, type, 2, P.out, size, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(ctx, BPE_ERR_CUDA, "head_logits: cuTensorMapEncodeTiled returned %d", (int)r);
    return BPE_OK;
}

// `p` itself where TMA can read it, else a copy in scratch (*copy, to be given back).
int aligned_rows(bpe_ctx *ctx, void **copy, const uint8_t *&p, uint64_t &stride, uint32_t rows, uint32_t dim) {
    if (rows == 1) stride = ((uint64_t)dim + 15) & ~15ull;
    if ((uintptr_t)p % 16 == 0 && stride % 16 == 0 && stride < (1ull << 40)) return BPE_OK;
    const uint32_t to = (dim + 15) & ~15u;
    void *q;
    int rc = head_scratch(ctx, (size_t)rows * to, &q);
    if (rc) return rc;
    *copy = q;
    const uint64_t want = ((uint64_t)rows * (to / 16) + 255) / 256;
    const uint32_t grid = (uint32_t)(want < (uint64_t)ctx->sm_count * 16 ? want : (uint64_t)ctx->sm_count * 16);
    k_head_align<<<grid, 256, 0, ctx->stream>>>(p, stride, rows, dim, (uint8_t *)q, to);
    BPE_CUDA(ctx, cudaGetLastError(), "head_logits align");
    p = (const uint8_t *)q;
    stride = to;
    return BPE_OK;
}

template <int kN, typename O>
int launch_few(bpe_ctx *ctx, const CUtensorMap &mw, const CUtensorMap &mx, const LogitsParams &P) {
    using F = Few<kN>;
    const uint32_t steps = (P.n_tok + kStep - 1) / kStep, each = (steps + ctx->sm_count - 1) / ctx->sm_count;
    auto k = k_logits_few<kN, O>;
    static std::atomic<uint64_t> devices{0};
    BPE_CUDA(ctx, allow_shared(k, ctx->device, F::kSmem, devices), "head_logits");
    k<<<(steps + each - 1) / each, F::kThreads, F::kSmem, ctx->stream>>>(mw, mx, P, each * kStep);
    BPE_CUDA(ctx, cudaGetLastError(), "head_logits launch");
    return BPE_OK;
}

template <typename O, int kCtas>
int launch_many(bpe_ctx *ctx, const CUtensorMap &mw, const CUtensorMap &mx, const CUtensorMap &mo, const LogitsParams &P) {
    using M = Many<kCtas>;
    auto k = k_logits_many<O, kCtas>;
    static std::atomic<uint64_t> devices{0};
    BPE_CUDA(ctx, allow_shared(k, ctx->device, M::kSmem, devices), "head_logits");
    const uint64_t n_tiles = (uint64_t)((P.n_rows + M::kRows - 1) / M::kRows) * ((P.n_tok + kManyToks - 1) / kManyToks);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctx->sm_count / kCtas * kCtas);
    cfg.blockDim = dim3(kManyThreads);
    cfg.dynamicSmemBytes = M::kSmem;
    cfg.stream = ctx->stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {kCtas, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = kCtas > 1 ? 1 : 0;
    // as many as run at once: a pair needs two free SMs of one GPC
    int &teams = ctx->head_teams[kCtas - 1];
    if (teams == 0) {
        if (kCtas == 1)
            teams = ctx->sm_count;
        else
            BPE_CUDA(ctx, cudaOccupancyMaxActiveClusters(&teams, k, &cfg), "head_logits");
        if (teams < 1) return fail(ctx, BPE_ERR_CUDA, "head_logits: no pair of CTAs fits");
    }
    cfg.gridDim = dim3((uint32_t)(n_tiles < (uint64_t)teams ? n_tiles : (uint64_t)teams) * kCtas);
    BPE_CUDA(ctx, cudaLaunchKernelEx(&cfg, k, mw, mx, mo, P), "head_logits launch");
    return BPE_OK;
}

template <typename O>
int launch(bpe_ctx *ctx, const uint8_t *x8, uint64_t x_stride, const uint8_t *w8, uint64_t w_stride, uint32_t dim, LogitsParams P) {
    const int n = P.n_rows <= 16 ? 16 : P.n_rows <= 32 ? 32 : P.n_rows <= 64 ? 64 : 0;
    P.tma_out = (uintptr_t)P.out % 16 == 0 && P.out_stride * sizeof(O) % 16 == 0 && P.out_stride * sizeof(O) < (1ull << 40);
    const uint64_t sms = (uint64_t)ctx->sm_count, row_tiles = (P.n_rows + 127) / 128, tok_tiles = (P.n_tok + kManyToks - 1) / kManyToks;
    const uint64_t singles = (row_tiles * tok_tiles + sms - 1) / sms, pairs = ((row_tiles + 1) / 2 * tok_tiles + sms / 2 - 1) / (sms / 2);
    // Pairs or single CTAs, by the rounds that each needs and what a round of pairs takes of one of single CTAs: 0.91 to
    // 0.94 measured over several rounds, more than all of it where there are few (2,000 x 4,352 x 1,024 f32: 19.1 us
    // against 17.3), 0.73 to 0.83 where rows start between lines of 128 bytes: loads cost more, and pairs load less.
    // 0.8 is the middle of eleven sizes of 300 to 1,100 rows, 60,000 to 250,000 tokens and 528 to 4,176 columns; at 272
    // columns it was 0.93 (640 x 100,000: 50 / 44 us).
    // In us, pairs / single CTAs: 512 x 250,000 x 1,024 120 / 129, x 1,040 147 / 175; 779 x 142,608 x 2,896 318 / 368;
    // 640 x 65,536 x 4,096 156 / 138; 384 x 65,536 x 4,096 103 / 98; 128 x 65,536 x 4,096 74 / 58.  An output that TMA
    // cannot write makes a tile's end longer than its loads (1,547 x 53,514 x 433: 120 / 108).  Up to 64 rows the few-row
    // kernel (64 x 65,536 x 4,096: 56 us against 53 by 128-row tiles, but 1,000 tokens fill 63 SMs instead of 4).
    const float share = P.tma_out && w_stride % kBlock ? 0.8f : singles >= 4 ? 0.95f : 1.05f;
    const bool pair = !n && (float)pairs * share < (float)singles;
    CUtensorMap mw, mx, mo = {};
    int rc;
    if ((rc = encode_map(ctx, &mw, w8, w_stride, P.n_tok, dim, n ? kStep : pair ? 128 : kManyToks)) ||
        (rc = encode_map(ctx, &mx, x8, x_stride, P.n_rows, dim, n ? n : 128)))
        return rc;
    if (n == 16) return launch_few<16, O>(ctx, mw, mx, P);
    if (n == 32) return launch_few<32, O>(ctx, mw, mx, P);
    if (n == 64) return launch_few<64, O>(ctx, mw, mx, P);
    if (P.tma_out && (rc = encode_out<O>(ctx, &mo, P))) return rc;
    return pair ? launch_many<O, 2>(ctx, mw, mx, mo, P) : launch_many<O, 1>(ctx, mw, mx, mo, P);
}

}  // namespace
}  // namespace bpe

using namespace bpe;

extern "C" int head_logits(bpe_ctx *ctx, const uint8_t *d_x8, uint64_t x8_stride, const float *d_xs, uint64_t xs_row_stride,
                           uint64_t xs_block_stride, const uint8_t *d_w8, uint64_t w8_stride, const float *d_ws,
                           uint64_t ws_row_stride, uint64_t ws_block_stride, uint32_t n_rows, uint32_t n_tok, uint32_t dim,
                           void *d_out, uint64_t out_stride, int out_type) {
    if (!ctx) return BPE_ERR_INVALID_ARG;
    if (!head_type_ok(out_type)) return fail(ctx, BPE_ERR_INVALID_ARG, "head_logits: unknown output type");
    if (dim == 0 || dim > BPE_HEAD_MAX_DIM || n_tok == 0 || n_tok > BPE_HEAD_MAX_TOKENS)
        return fail(ctx, BPE_ERR_INVALID_ARG, "head_logits: %u tokens of %u columns", n_tok, dim);
    if (n_rows == 0) return BPE_OK;
    if (n_rows > BPE_HEAD_MAX_TOKENS) return fail(ctx, BPE_ERR_INVALID_ARG, "head_logits: %u rows", n_rows);
    if (!d_x8 || !d_xs || !d_w8 || !d_ws || !d_out) return fail(ctx, BPE_ERR_INVALID_ARG, "head_logits: null pointer");
    if ((n_rows > 1 && (x8_stride < dim || out_stride < n_tok)) || (n_tok > 1 && w8_stride < dim))
        return fail(ctx, BPE_ERR_INVALID_ARG, "head_logits: a row stride is below its row's length");
    BPE_CUDA(ctx, cudaSetDevice(ctx->device), "cudaSetDevice");
    int rc;
    uint32_t *status;
    if ((rc = head_status(ctx, &status))) return rc;
    void *copy_x = nullptr, *copy_w = nullptr;
    rc = aligned_rows(ctx, &copy_x, d_x8, x8_stride, n_rows, dim);
    if (!rc) rc = aligned_rows(ctx, &copy_w, d_w8, w8_stride, n_tok, dim);
    const LogitsParams P{d_xs, d_ws, d_out, xs_row_stride, xs_block_stride, ws_row_stride, ws_block_stride, out_stride,
                         n_rows, n_tok, (dim + kBlock - 1) / kBlock, false, status, ctx->test_stall_head};
    if (!rc)
        rc = out_type == BPE_F32    ? launch<float>(ctx, d_x8, x8_stride, d_w8, w8_stride, dim, P)
             : out_type == BPE_BF16 ? launch<__nv_bfloat16>(ctx, d_x8, x8_stride, d_w8, w8_stride, dim, P)
                                    : launch<__half>(ctx, d_x8, x8_stride, d_w8, w8_stride, dim, P);
    int freed = head_scratch_free(ctx, copy_x);
    if (!freed) freed = head_scratch_free(ctx, copy_w);
    return rc ? rc : freed;
}
