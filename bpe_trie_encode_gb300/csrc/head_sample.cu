// head_sample.cu -- temperature, top-k, top-p, min-p and the draw of one id
// per row from a given random number.
//
// With m the row's largest logit, z = (l - m) / T and the whole numbers
// w = floor(exp(z) 2^40): sums of w are exact, so neither the split of a row
// over threads and CTAs nor the order of atomics changes an answer.  The three
// filters keep a prefix of the tokens ordered by logit (then by id), so that
// one cut -- a last kept token -- describes what is kept, and the draw is a
// search for a running sum in order of ids.
//
// A row is read once, into the shared memory of one CTA (up to 46,000 tokens of
// 32 bits, 92,000 of 16), or of a cluster of up to 8 where it does not fit or
// where SMs are idle: a barrier of a cluster costs over 1,000 cycles and a row
// needs six, so a split never takes an SM from another row.  The cut is found by histograms over -z in fixed
// point: 4 buckets per unit, then 128 of the bucket that holds the cut, and so
// on until at most 128 tokens are left, which are ranked by comparing all pairs.
//
// What bounds it is not the read but the work per logit, about 20 instructions
// for an exponential and an exact weight, 26 more with two shared-memory
// atomics for the first histogram; a small top-k needs neither (2 instructions)
// and is bound by the latency of its steps.  Measured: 4,096 rows of 4,352 bf16
// without filters 25 us (1.4 TB/s; 34 instructions a logit, 70% of the issue
// slots); 256 x 65,536 bf16 with all filters 26 us (1.3 TB/s); 61 x 250,000 f32,
// top-p over flat rows, 111 to 119 us by where its clusters land (100
// instructions a logit, 41% of the issue slots, barriers the first of its
// stalls); 1 x 32,256 f32, top-p, 14 to 16 us.
#include "head.cuh"

#include "device.cuh"
#include "internal.h"

namespace bpe {
namespace {

constexpr int kSampThreads = 512;
constexpr float kOne = 1099511627776.0f;   // 2^40

typedef unsigned long long u64;

struct SampleParams {
    const void *logits;
    uint64_t stride;
    uint32_t n_tok;
    int type;
    const float *u;
    head_filters f;
    int32_t *ids;
    float *logprob;
};

// Logits as whole numbers of the same order (a NaN as -infinity, -0 as 0).
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    const uint32_t k = b & 0x80000000u ? ~b : b | 0x80000000u;
    return v != v ? kKeyNegInf : k;
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

__device__ __forceinline__ float z_of(float v, float top, float inv_t) {
    return v == top ? 0.0f : __fmul_rn(v - top, inv_t);
}

// w = floor(e 2^40) in two parts of 20 bits, for 0 <= e <= 1: additions that round towards zero leave the whole part
// of e 2^20, then of its rest times 2^20, in the low bits of a float between 2^23 and 2^24.
constexpr uint32_t kWhole = 0x4B000000u;   // 2^23
struct Parts { uint32_t hi, lo; };
__device__ __forceinline__ Parts parts_of(float e) {
    const float t = __fmaf_rz(e, 0x1p20f, 0x1p23f);
    const float l = __fmaf_rz(fmaf(e, 0x1p20f, 0x1p23f - t), 0x1p20f, 0x1p23f);
    return {__float_as_uint(t) - kWhole, __float_as_uint(l) - kWhole};
}
// Sums of both parts; what the 2^23 of each addition adds is taken off at the end.
struct PartSum {
    uint32_t hi = 0, lo = 0;
    __device__ __forceinline__ void add(float e) {
        const float t = __fmaf_rz(e, 0x1p20f, 0x1p23f);
        hi += __float_as_uint(t);
        lo += __float_as_uint(__fmaf_rz(fmaf(e, 0x1p20f, 0x1p23f - t), 0x1p20f, 0x1p23f));
    }
    __device__ __forceinline__ u64 value(uint32_t n) const { return ((u64)(hi - n * kWhole) << 20) + (lo - n * kWhole); }
};
__device__ __forceinline__ u64 join(uint32_t hi, uint32_t lo) { return ((u64)hi << 20) + lo; }
__device__ __forceinline__ u64 weight(float e) {
    const Parts p = parts_of(e);
    return join(p.hi, p.lo);
}

// ------------------------------------------------- rows in shared memory ---
constexpr int kBuckets = 128;
constexpr float kCodeScale = -0x1p27f;     // -z as a whole number
constexpr int kList = 128;                 // tokens that are ranked pair by pair
constexpr int kMaxTeam = 8;
constexpr size_t kMaxShared = 232448, kSmShared = 233472;   // of a CTA, of an SM
constexpr int kSmallK = 256, kSmall = 512; // top-k up to kSmallK works on a list of up to kSmall tokens
constexpr int kRowCtas = 12;               // of 128 threads, an SM
constexpr int kNear = 256;                 // buckets of 1/8 below the largest logit, for that list

struct __align__(16) Entry { uint32_t key, idx; u64 w; };

// kTeam: the row's CTAs are several.  kCut: with top-k or top-p.
template <int kThreads, bool kTeam, bool kCut> struct SampleShared {
    static constexpr int kCopies = kThreads / 32;   // of a histogram, by thread: no more than 4,095 tokens meet in one
    uint32_t lo[kCut ? kBuckets * kCopies : 4], hi[kCut ? kBuckets * kCopies : 4];
    u64 sum[2][kTeam ? kBuckets : 1];      // this CTA's histogram, read by the whole cluster
    u64 all[!kCut ? 2 : kTeam ? kNear : kBuckets];     // the row's
    uint32_t near_n[kCut ? kNear : 4];                // groups of logits by their largest
    u64 slot[2][kMaxTeam];                 // a value from each CTA of the cluster
    u64 red[32];
    Entry mine[kTeam ? kList : 1];         // tokens of the last bucket: this CTA's, read by the whole cluster
    union {
        Entry list[kCut ? kList : 1];      // and the row's
        u64 small[kCut ? kSmall : 2];                 // logit and id of the largest tokens: this CTA's, read by the first CTA
    };
    uint32_t list_n, small_n;
    u64 pick[4];                           // bucket found, sums above and in it, this CTA's sum above it
    u64 goal;
    float cut_v;                           // the last kept token
    uint32_t cut_idx;
    uint4 row[1];                          // the CTA's logits as they are, 16 bytes at a time
};

__device__ __forceinline__ uint32_t far_addr(const void *p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void far_store(void *p, uint32_t rank, u64 v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(far_addr(p, rank)), "l"(v) : "memory");
}
__device__ __forceinline__ void far_store(uint32_t *p, uint32_t rank, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(far_addr(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ u64 far_load(const u64 *p, uint32_t rank) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(far_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t far_load(const uint32_t *p, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(far_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint4 far_load(const Entry *p, uint32_t rank) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(far_addr(p, rank)) : "memory");
    return v;
}
// The counter at this shared address += v, where v is not 0; without a branch around it.
__device__ __forceinline__ void count_up(uint32_t at, uint32_t v) {
    asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %1, 0;\n@p red.shared.add.u32 [%0], %1;\n}" ::"r"(at), "r"(v) : "memory");
}

__device__ __forceinline__ u64 warp_sum(u64 v) {   // of values below 2^63, by parts of 22 bits
    const uint32_t a = __reduce_add_sync(kFull, (uint32_t)v & 0x3FFFFFu);
    const uint32_t b = __reduce_add_sync(kFull, (uint32_t)(v >> 22) & 0x3FFFFFu);
    const uint32_t c = __reduce_add_sync(kFull, (uint32_t)(v >> 44));
    return a + ((u64)b << 22) + ((u64)c << 44);
}
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {   // inclusive
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const u64 o = __shfl_up_sync(kFull, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// kHalf: logits of 16 bits.
template <bool kHalf, int kThreads, bool kTeam, bool kCut>
struct Sampler {
    using Shared = SampleShared<kThreads, kTeam, kCut>;
    static constexpr int kWarps = kThreads / 32, kCopies = Shared::kCopies;
    static constexpr int kVec = kHalf ? 8 : 4;   // logits in 16 bytes
    Shared &S;
    const SampleParams &P;
    const uint4 *data;      // the CTA's logits
    uint32_t rank, team;    // this CTA among the row's
    uint32_t first, count;  // its tokens
    uint32_t g0, g1;        // a thread's groups of 16 bytes: contiguous, an odd number, so that no two lanes' meet in a bank
    int lane, warp, turn;
    float top, temp, inv_t;
    float cut_v;
    uint32_t cut_idx;

    __device__ __forceinline__ uint32_t members() const { return kTeam ? team : 1; }
    __device__ __forceinline__ void sync() const {
        __syncwarp();
        if (members() == 1)
            __syncthreads();
        else
            asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    __device__ __forceinline__ float decode(uint32_t half) const {   // 16 bits of either type
        return P.type == BPE_BF16 ? __uint_as_float(half << 16) : __half2float(__ushort_as_half((unsigned short)half));
    }
    __device__ __forceinline__ float logit(uint32_t i) const {       // of the CTA's token i
        if (kHalf) return decode(((const unsigned short *)data)[i]);
        return ((const float *)data)[i];
    }
    __device__ __forceinline__ void unpack(const uint4 &q, float (&v)[kVec]) const {
        if (!kHalf) {
            v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
        } else {
            const uint32_t w[4] = {q.x, q.y, q.z, q.w};
            if (P.type == BPE_BF16) {
#pragma unroll
                for (int i = 0; i < 4; i++) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            } else {
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float2 f = __half22float2(*(const __half2 *)&w[i]);
                    v[2 * i] = f.x, v[2 * i + 1] = f.y;
                }
            }
        }
    }
    // f(first of the tokens, logits) for this thread's groups; those past the end are -infinity
    template <typename F> __device__ __forceinline__ void groups(F f) const {
#pragma unroll (kHalf ? 1 : 2)
        for (uint32_t g = g0; g < g1; g++) {
            float v[kVec];
            unpack(data[g], v);
            f(g * kVec, v);
        }
    }
    // the largest of a group, NaN aside
    __device__ __forceinline__ float most(const uint4 &q) const {
        if (!kHalf)
            return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
        if (P.type == BPE_BF16) {
            const __nv_bfloat162 *h = (const __nv_bfloat162 *)&q;
            const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
            return __bfloat162float(__hmax(m.x, m.y));
        }
        const __half2 *h = (const __half2 *)&q;
        const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return __half2float(__hmax(m.x, m.y));
    }
    // f(i, logit) for this thread's tokens with logits in [low, high]: few, so that most groups end with their largest
    template <typename F> __device__ __forceinline__ void few(float low, float high, F f) const {
#pragma unroll 2
        for (uint32_t g = g0; g < g1; g++) {
            const uint4 q = data[g];
            if (most(q) >= low) {
                float v[kVec];
                unpack(q, v);
#pragma unroll
                for (int j = 0; j < kVec; j++)
                    if (v[j] >= low && v[j] <= high) f(g * kVec + j, v[j]);
            }
        }
    }
    // f(i, logit) for this thread's groups whose largest is `low` at least
    template <typename F> __device__ __forceinline__ void some(float low, F f) const {
#pragma unroll (kHalf ? 1 : 2)
        for (uint32_t g = g0; g < g1; g++) {
            const uint4 q = data[g];
            if (most(q) >= low) {
                float v[kVec];
                unpack(q, v);
#pragma unroll
                for (int j = 0; j < kVec; j++) f(g * kVec + j, v[j]);
            }
        }
    }
    // Bounds of the logits whose z is in [z0, z1]: wider by more than all rounding (z is above -33).
    __device__ __forceinline__ float least_logit(float z0) const {
        return top + (z0 - 1e-3f) * temp - 1e-6f * (fabsf(top) + 40.0f * temp);
    }
    __device__ __forceinline__ float most_logit(float z1) const {
        return z1 > -2e-3f ? INFINITY : top + (z1 + 1e-3f) * temp + 1e-6f * (fabsf(top) + 40.0f * temp);
    }
    // f(i, logit) for this thread's tokens
    template <typename F> __device__ __forceinline__ void each(F f) const {
#pragma unroll 1
        for (uint32_t g = g0; g < g1; g++) {
            float v[kVec];
            unpack(data[g], v);
#pragma unroll
            for (int j = 0; j < kVec; j++) f(g * kVec + j, v[j]);
        }
    }
    // z, or -31.75 where nothing can be drawn; NaN too
    __device__ __forceinline__ float z_at(float v) const { return fmaxf(__fmul_rn(v - top, inv_t), -31.75f); }
    __device__ __forceinline__ uint32_t code_at(float z) const { return __float2uint_rz(z * kCodeScale); }
    __device__ __forceinline__ u64 weight_at(float v) const { return weight(expf(z_at(v))); }

    // Before a row: a thread's share of it, and clear counters.
    __device__ __forceinline__ void begin_row() {
        const uint32_t n = (count + kVec - 1) / kVec, span = ((n + kThreads - 1) / kThreads) | 1;
        g0 = min(n, threadIdx.x * span), g1 = min(n, (threadIdx.x + 1) * span);
        lane = threadIdx.x & 31, warp = threadIdx.x >> 5, turn = 0;
        if (kCut) {
            for (int i = threadIdx.x; i < kBuckets * kCopies; i += kThreads) S.lo[i] = S.hi[i] = 0;
            for (int i = threadIdx.x; i < kNear; i += kThreads) S.near_n[i] = 0;
            if (threadIdx.x == 0) S.small_n = 0;
        }
    }

    // One value per CTA to every CTA of the row; all threads of the CTA hold `v`.
    __device__ __forceinline__ void exchange(u64 v) {
        turn ^= 1;
        if (threadIdx.x < members()) far_store(&S.slot[turn][rank], threadIdx.x, v);
        sync();
    }
    __device__ __forceinline__ uint32_t max_row(uint32_t v) {
        v = __reduce_max_sync(kFull, v);
        __syncthreads();
        if (lane == 0) S.red[warp] = v;
        __syncthreads();
        v = __reduce_max_sync(kFull, lane < kWarps ? (uint32_t)S.red[lane] : 0);
        if (members() == 1) return v;
        exchange(v);
        v = 0;
        for (uint32_t r = 0; r < members(); r++) v = max(v, (uint32_t)S.slot[turn][r]);
        return v;
    }
    // The CTA's sum; the warps' stay in S.red.
    __device__ __forceinline__ u64 sum_cta(u64 v) {
        v = warp_sum(v);
        __syncthreads();
        if (lane == 0) S.red[warp] = v;
        __syncthreads();
        return warp_sum(lane < kWarps ? S.red[lane] : 0);
    }
    // The row's sum of the CTAs' sums; `before`: of the CTAs before this one.
    __device__ __forceinline__ u64 sum_ctas(u64 mine, u64 &before) {
        before = 0;
        if (members() == 1) return mine;
        exchange(mine);
        u64 total = 0;
        for (uint32_t r = 0; r < members(); r++) {
            const u64 x = S.slot[turn][r];
            before += r < rank ? x : 0;
            total += x;
        }
        return total;
    }
    __device__ __forceinline__ u64 sum_row(u64 v) {
        u64 before;
        return sum_ctas(sum_cta(v), before);
    }

    // The token, in order of ids, at which the running sum of value(i, logit) passes t; the lane that holds it calls
    // found(i).  own: this thread's sum; S.red holds the warps', `mine` is the CTA's, `before` the CTAs' before it.
    template <typename V, typename F>
    __device__ __forceinline__ void locate(V value, u64 own, u64 t, u64 before, u64 mine, F found) const {
        if (t < before || t - before >= mine) return;
        t -= before;
        const u64 w = lane < kWarps ? S.red[lane] : 0, run = warp_scan(w, lane);
        if (__ffs(__ballot_sync(kFull, run > t)) - 1 != warp) return;
        t -= __shfl_sync(kFull, run - w, warp);
        const u64 upto = warp_scan(own, lane);
        const int who = __ffs(__ballot_sync(kFull, upto > t)) - 1;
        t -= __shfl_sync(kFull, upto - own, who);
        const uint32_t i0 = __shfl_sync(kFull, g0, who) * kVec, i1 = __shfl_sync(kFull, g1, who) * kVec;
        for (uint32_t i = i0 + lane; i - lane < i1; i += 32) {   // the thread's tokens, a lane each
            const u64 v = i < i1 ? value(i, logit(i)) : 0, s = warp_scan(v, lane);
            const unsigned past = __ballot_sync(kFull, s > t);
            if (past) {
                if (lane == __ffs(past) - 1) found(i);
                return;
            }
            t -= __shfl_sync(kFull, s, 31);
        }
    }

    __device__ __forceinline__ bool in_cut(uint32_t i, float v) const {
        return (v > cut_v) | ((v == cut_v) & (first + i <= cut_idx));
    }
    __device__ __forceinline__ u64 kept(uint32_t i, float v, u64 least) const {
        const u64 w = in_cut(i, v) ? weight_at(v) : 0;
        return w >= least ? w : 0;
    }
    // This thread's kept mass: at most 104 tokens, so the parts' sums stay below 2^32.
    __device__ __forceinline__ u64 mass(u64 least) const {
        PartSum sum;
        if (cut_v == -INFINITY && !least) {   // everything
            each([&](uint32_t, float v) { sum.add(expf(z_at(v))); });
            return sum.value((g1 - g0) * kVec);
        }
        return least ? mass_above<true>(least) : mass_above<false>(0);
    }
    template <bool kLeastOn> __device__ __forceinline__ u64 mass_above(u64 least) const {
        PartSum sum;
        const float floor_v = kLeastOn ? fmaxf(cut_v, least_logit(logf((float)least * 0x1p-40f))) : cut_v;
        uint32_t n = 0;
#pragma unroll (kHalf ? 1 : 2)
        for (uint32_t g = g0; g < g1; g++) {
            const uint4 q = data[g];
            if (most(q) >= floor_v) {
                float v[kVec];
                unpack(q, v);
#pragma unroll
                for (int j = 0; j < kVec; j++) {
                    float e = expf(z_at(v[j]));
                    e = in_cut(g * kVec + j, v[j]) ? e : 0.0f;
                    if (kLeastOn) e = weight(e) < least ? 0.0f : e;
                    sum.add(e);
                }
                n += kVec;
            }
        }
        return sum.value(n);
    }
    __device__ __forceinline__ void read_cut() { cut_v = S.cut_v, cut_idx = S.cut_idx; }

    // The last token kept when tokens are taken in order (largest logit, then lowest id) until the sum of their
    // values -- 1, or the weight -- reaches the target: `target`, or with share >= 0 that share of the whole sum, and
    // at least 1.  Where the whole sum is below the target, everything is kept and the cut stays.  kFirst: the
    // histogram is clear.  With kMass, *total and *mine become the row's kept sum and this CTA's, unless false is
    // returned.
    template <bool kMass, bool kFirst>
    __device__ __forceinline__ bool select(u64 target, double share, u64 *total = nullptr, u64 *mine = nullptr) {
        u64 above = 0, own = 0;
        uint32_t low = 0;
        int shift = 25, buckets = kBuckets, copies = kCopies;
        // After the first level the bucket's tokens, where they fit, are listed in the upper half of the histogram's
        // place, and the levels that follow (4 copies, in the lower half) read only them.
        constexpr bool kPick = kThreads >= 256;
        uint32_t *const picked = S.hi, *upper = S.hi;
        uint32_t n_pick = ~0u;
        auto in_range = [&](uint32_t width, auto f) {
            if (n_pick != ~0u) {
                for (uint32_t j = threadIdx.x; j < n_pick; j += kThreads) f(picked[j], logit(picked[j]));
            } else {
                few(least_logit((float)(low + width) / kCodeScale), most_logit((float)low / kCodeScale), f);
            }
        };
        for (int level = 0;; level++) {
            // histogram of the codes in [low, low + (buckets << shift))
            if (!kFirst || level > 0) {
                for (int i = threadIdx.x; i < buckets * copies; i += kThreads) {
                    S.lo[i] = 0;
                    if (kMass) upper[i] = 0;
                }
            }
            if (threadIdx.x == 0) S.list_n = 0, S.pick[0] = ~0ull;
            __syncthreads();
            const int copy = threadIdx.x & (copies - 1);
            const uint32_t lo_at = (uint32_t)__cvta_generic_to_shared(S.lo + copy), hi_at = (uint32_t)__cvta_generic_to_shared(upper + copy);
            if (level == 0) {
                // floor(-4 z), the code's upper bits, lies in the low bits of a sum that rounds towards zero; times the
                // size of a bucket, the 2^23 above it is taken off the addresses
                constexpr uint32_t kSize = kCopies * 4, kOff = kWhole * kSize;
                each([&](uint32_t, float v) {
                    const float z = z_at(v);
                    const uint32_t at = __float_as_uint(__fmaf_rz(z, -4.0f, 0x1p23f)) * kSize - kOff;
                    if (kMass) {
                        const Parts p = parts_of(expf(z));
                        count_up(lo_at + at, p.lo);
                        count_up(hi_at + at, p.hi);
                    } else {
                        count_up(lo_at + at, z > -28.0f);
                    }
                });
            } else {
                const uint32_t width = ((uint32_t)buckets << shift) - 1;
                in_range(width, [&](uint32_t, float v) {
                    const float z = z_at(v);
                    const uint32_t c = code_at(z) - low;
                    if (c <= width) {
                        const Parts p = kMass ? parts_of(expf(z)) : Parts{0, 1};
                        const uint32_t at = (c >> shift) * copies * 4;
                        count_up(lo_at + at, p.lo);
                        if (kMass) count_up(hi_at + at, p.hi);
                    }
                });
            }
            __syncthreads();
            u64 *sum = members() == 1 ? S.all : S.sum[level & 1];
            for (int i = threadIdx.x; i < buckets * 4; i += kThreads) {   // four lanes a bucket; whole warps: 16 buckets at least
                const int b = i >> 2;
                u64 v = 0;
                for (int c = 0; c < copies; c += 4) {
                    const int a = b * copies + (((i & 3) + c + b * 4) & (copies - 1));
                    v += join(kMass ? upper[a] : 0, S.lo[a]);
                }
                v += __shfl_xor_sync(kFull, v, 1);
                v += __shfl_xor_sync(kFull, v, 2);
                if ((i & 3) == 0) sum[b] = v;
            }
            sync();
            if (members() > 1) {
                for (int b = threadIdx.x; b < buckets; b += kThreads) {
                    u64 v[kMaxTeam], s = 0;
#pragma unroll
                    for (int r = 0; r < kMaxTeam; r++) v[r] = (uint32_t)r < members() ? far_load(sum + b, r) : 0;
#pragma unroll
                    for (int r = 0; r < kMaxTeam; r++) s += v[r];
                    S.all[b] = s;
                }
                __syncthreads();
            }
            // largest logits first, the bucket at which the running sum reaches the target
            if (warp == 0) {
                constexpr int kPer = kBuckets / 32;
                u64 v[kPer], s = 0, m = 0;
#pragma unroll
                for (int j = 0; j < kPer; j++) {
                    const int b = lane * kPer + j;
                    v[j] = b < buckets ? S.all[b] : 0;
                    s += v[j];
                    if (kMass && members() > 1 && b < buckets) m += sum[b];
                }
                u64 run = warp_scan(s, lane), part = kMass && members() > 1 ? warp_scan(m, lane) - m : 0;
                if (level == 0 && share >= 0.0) {
                    const double x = share * (double)__shfl_sync(kFull, run, 31);
                    target = x > 1.0 ? (u64)x : 1;
                }
                run = above + run - s;
#pragma unroll
                for (int j = 0; j < kPer; j++) {
                    const int b = lane * kPer + j;
                    if (run < target && target <= run + v[j]) {
                        S.pick[0] = b;
                        S.pick[1] = run;
                        S.pick[2] = v[j];
                        S.pick[3] = members() > 1 ? part : run;
                    }
                    run += v[j];
                    if (kMass && members() > 1 && b < buckets) part += sum[b];
                }
                if (lane == 0) S.goal = target;
            }
            __syncthreads();
            if (S.pick[0] == ~0ull) return false;   // at level 0: less than the target in all
            target = S.goal;
            low += (uint32_t)S.pick[0] << shift;
            above = S.pick[1];
            own = members() > 1 ? own + S.pick[3] : above;
            // are the bucket's tokens few?  By weight: an estimate, and the list says when it was wrong.
            u64 about = S.pick[2];
            if (kMass) {
                const float e = expf((float)low * (1.0f / kCodeScale));
                about = e > 0x1p-38f ? (u64)((float)about / (e * kOne)) : 0;
            }
            if (about <= kList || shift == 0) {
                const uint32_t width = (1u << shift) - 1;
                Entry *to = members() == 1 ? S.list : S.mine;
                in_range(width, [&](uint32_t i, float v) {
                    if (code_at(z_at(v)) - low <= width) {
                        const uint32_t n = atomicAdd(&S.list_n, 1u);
                        if (n < kList) to[n] = Entry{key_of(v), first + i, weight_at(v)};
                    }
                });
                sync();
                uint32_t n = S.list_n;
                if (members() > 1) {   // every CTA's to one list
                    uint32_t c = (uint32_t)lane < members() ? far_load(&S.list_n, lane) : 0;
                    const uint32_t end = warp_incl_sum(c, lane);
                    n = __shfl_sync(kFull, end, 31);
                    for (uint32_t i = threadIdx.x; i < ((n + 31) & ~31u) && n <= kList; i += kThreads) {
                        uint32_t from = 0, begin = 0;   // the CTA whose part holds place i
#pragma unroll
                        for (int r = 0; r < kMaxTeam - 1; r++) {
                            const uint32_t e = __shfl_sync(kFull, end, r);
                            if ((uint32_t)r < members() && i >= e) from = r + 1, begin = e;
                        }
                        if (i < n) *reinterpret_cast<uint4 *>(&S.list[i]) = far_load(&S.mine[i - begin], from);
                    }
                    __syncthreads();
                }
                if (n <= kList) {
                    // four lanes a token add up what comes before it
                    for (uint32_t i = threadIdx.x / 4; i < ((n + 7) & ~7u); i += kThreads / 4) {
                        const Entry x = S.list[min(i, n - 1)];
                        u64 run = 0, here = 0;
                        for (uint32_t j = lane & 3; j < n; j += 4) {
                            const Entry y = S.list[j];
                            const bool before = y.key > x.key || (y.key == x.key && y.idx < x.idx);
                            if (before) run += kMass ? y.w : 1;
                            if (kMass && members() > 1 && (before || j == i) && y.idx - first < count) here += y.w;
                        }
                        run += __shfl_xor_sync(kFull, run, 1);
                        run += __shfl_xor_sync(kFull, run, 2);
                        if (kMass && members() > 1) {
                            here += __shfl_xor_sync(kFull, here, 1);
                            here += __shfl_xor_sync(kFull, here, 2);
                        }
                        run += above;
                        const u64 upto = run + (kMass ? x.w : 1);
                        if (i < n && run < target && target <= upto) {
                            S.cut_v = key_value(x.key);
                            S.cut_idx = x.idx;
                            S.pick[1] = upto;
                            S.pick[3] = members() > 1 ? own + here : upto;
                        }
                    }
                    __syncthreads();
                    if (kMass && total) *total = S.pick[1], *mine = S.pick[3];
                    return true;
                }
                if (shift == 0) break;   // over kList tokens of one code
                sync();                  // list_n has been read by all
            }
            __syncthreads();             // what was found has been read by all
            if (kPick && level == 0) {   // z in (z0, z1] is the bucket
                const float z0 = (float)(low + (1u << shift)) / kCodeScale, z1 = (float)low / kCodeScale;
                const float v0 = least_logit(z0);
                uint32_t mine_n = 0;
                auto in = [&](float v) { const float z = __fmul_rn(v - top, inv_t); return (z > z0) & (z <= z1); };
                some(v0, [&](uint32_t, float v) { mine_n += in(v); });
                const uint32_t upto = warp_incl_sum(mine_n, lane);
                if (lane == 31) S.red[warp] = upto;
                __syncthreads();
                const uint32_t w = lane < kWarps ? (uint32_t)S.red[lane] : 0, run = warp_incl_sum(w, lane);
                const uint32_t n = __shfl_sync(kFull, run, 31);
                if (n <= kBuckets * kCopies) {
                    uint32_t at = __shfl_sync(kFull, run - w, warp) + upto - mine_n;
                    some(v0, [&](uint32_t i, float v) {
                        if (in(v)) picked[at++] = i;
                    });
                    n_pick = n;
                    copies = 4;
                    upper = S.lo + kBuckets * 4;
                }
                __syncthreads();
            }
            buckets = shift >= 7 ? 128 : 1 << shift;
            shift = shift >= 7 ? shift - 7 : 0;
        }
        // tokens of one code: by logit, then by id
        auto in = [&](float v) { return code_at(z_at(v)) == low; };
        auto value = [&](float v) -> u64 { return kMass ? weight_at(v) : 1; };
        uint32_t big = 0, small = 0;
        each([&](uint32_t, float v) {
            if (in(v)) {
                big = max(big, key_of(v));
                small = max(small, ~key_of(v));
            }
        });
        big = max_row(big);
        small = ~max_row(small);
        uint32_t at = small;
        u64 need = target - above;
        if (big != small) {          // logits that differ by less than a code
            at = 0;
            for (int bit = 31; bit >= 0; bit--) {
                const uint32_t c = at | 1u << bit;
                u64 m = 0;
                each([&](uint32_t, float v) { m += in(v) && key_of(v) >= c ? value(v) : 0; });
                if (sum_row(m) >= need) at = c;
            }
            u64 m = 0;
            each([&](uint32_t, float v) { m += in(v) && key_of(v) > at ? value(v) : 0; });
            need -= sum_row(m);
        }
        const float last = key_value(at);
        const u64 w = value(last);
        need = (need + w - 1) / w;   // that many of the logit `last`
        auto one = [&](uint32_t, float v) -> u64 { return v == last; };
        u64 m = 0, before;
        each([&](uint32_t i, float v) { m += one(i, v); });
        const u64 part = sum_cta(m);
        sum_ctas(part, before);
        locate(one, m, need - 1, before, part, [&](uint32_t i) {
            for (uint32_t r = 0; r < members(); r++) far_store(&S.cut_idx, r, first + i);
        });
        if (threadIdx.x == 0) S.cut_v = last;
        sync();
        return false;
    }

    // top-k up to kSmallK, with what follows it, on a list: the k-th largest of the groups' largest logits (in short
    // rows, of all logits) is a lower bound of the k-th largest logit, and few tokens lie above it.  Only they need an
    // exponential.  Returns false, with nothing done, where the list would not do.
    __device__ __forceinline__ bool small_list(uint32_t k, float p, u64 least, uint32_t row) {
        const float scale = inv_t * 8.0f;
        auto near = [&](float v) { return __fmul_rn(top - v, scale); };   // grows as v falls
        auto file = [&](float v) {
            const float x = near(v);
            if (x < (float)kNear) atomicAdd(&S.near_n[(int)x], 1u);
        };
        if (kThreads >= 512) {
            // a k above the number of groups (512 tokens of 16 bits have 64) finds no bound here and goes on to select
            for (uint32_t g = g0; g < g1; g++) file(most(data[g]));
        } else {
            each([&](uint32_t, float v) { file(v); });
        }
        sync();
        if (members() > 1) {
            for (int b = threadIdx.x; b < kNear; b += kThreads) {
                uint32_t v = 0;
                for (uint32_t r = 0; r < members(); r++) v += far_load(S.near_n + b, r);
                S.all[b] = v;
            }
            __syncthreads();
        }
        if (warp == 0) {
            constexpr int kPer = kNear / 32;
            uint32_t v[kPer], s = 0, edge = ~0u;
#pragma unroll
            for (int j = 0; j < kPer; j++)
                s += v[j] = members() > 1 ? (uint32_t)S.all[lane * kPer + j] : S.near_n[lane * kPer + j];
            uint32_t run = warp_incl_sum(s, lane) - s;
#pragma unroll
            for (int j = 0; j < kPer; j++) {
                if (run < k && k <= run + v[j]) edge = lane * kPer + j + 1;
                run += v[j];
            }
            edge = __reduce_min_sync(kFull, edge);
            if (lane == 0) S.pick[0] = edge;
        }
        __syncthreads();
        if ((uint32_t)S.pick[0] == ~0u) return false;
        const float edge = least_logit((float)(uint32_t)S.pick[0] * -0.125f);
        few(edge, INFINITY, [&](uint32_t i, float v) {
            const uint32_t n = atomicAdd(&S.small_n, 1u);
            if (n < kSmall) S.small[n] = (u64)key_of(v) << 32 | (uint32_t)~(first + i);
        });
        sync();
        uint32_t n = S.small_n;
        if (members() > 1) {
            uint32_t c = (uint32_t)lane < members() ? far_load(&S.small_n, lane) : 0;
            n = __reduce_add_sync(kFull, c);
            if (n <= kSmall && rank == 0) {   // the other CTAs' behind this one's
                uint32_t at = S.small_n;
                for (uint32_t r = 1; r < members(); r++) {
                    const uint32_t m = __shfl_sync(kFull, c, r);
                    for (uint32_t i = threadIdx.x; i < m; i += kThreads) S.small[at + i] = far_load(S.small + i, r);
                    at += m;
                }
            }
            sync();           // the other CTAs end here
        }
        if (n > kSmall) return false;
        if (rank != 0) return true;
        u64 *order = (u64 *)S.lo, *heavy = order + kSmallK;   // in the histogram's place
        static_assert(sizeof(S.lo) + sizeof(S.hi) >= 2 * kSmallK * sizeof(u64), "room for the sorted list");
        // sorted: a token's place is the number of larger ones, counted by four lanes
        for (uint32_t i = threadIdx.x / 4; i < ((n + 7) & ~7u); i += kThreads / 4) {
            const u64 y = S.small[min(i, n - 1)];
            uint32_t place = 0;
#pragma unroll 4
            for (uint32_t j = lane & 3; j < n; j += 4) place += S.small[j] > y;
            place += __shfl_xor_sync(kFull, place, 1);
            place += __shfl_xor_sync(kFull, place, 2);
            if (i < n && place < k && (lane & 3) == 0) {
                order[place] = y;
                heavy[place] = weight_at(key_value((uint32_t)(y >> 32)));
            }
        }
        __syncthreads();
        n = min(n, k);
        if (warp == 0) {   // 8 tokens a lane
            constexpr int kPer = kSmallK / 32;
            u64 w[kPer], s = 0;
#pragma unroll
            for (int j = 0; j < kPer; j++) {
                w[j] = (uint32_t)(lane * kPer + j) < n ? heavy[lane * kPer + j] : 0;
                s += w[j];
            }
            const u64 upto = warp_scan(s, lane);
            u64 edge = ~0ull;
            if (p < 1.0f) {
                const double y = (double)p * (double)__shfl_sync(kFull, upto, 31);
                edge = y > 1.0 ? (u64)y : 1;
            }
            u64 run = upto - s, total = 0;
            uint32_t keep = 0;
#pragma unroll
            for (int j = 0; j < kPer; j++) {
                const bool in = w[j] > 0 && run < edge;
                run += w[j];
                if (!(in && w[j] >= least)) w[j] = 0;
                if (in) keep++;
                total += w[j];
                if ((uint32_t)(lane * kPer + j) < n) heavy[lane * kPer + j] = w[j];
            }
            keep = __reduce_add_sync(kFull, keep);
            total = warp_sum(total);
            if (lane == 0) S.pick[1] = keep, S.pick[2] = total, S.goal = goal_of(row, total);
        }
        __syncthreads();
        const uint32_t keep = (uint32_t)S.pick[1];
        const u64 total = S.pick[2], t = S.goal;
        for (uint32_t i = threadIdx.x / 4; i < ((keep + 7) & ~7u); i += kThreads / 4) {
            const uint32_t mine = (uint32_t)order[min(i, keep - 1)];   // ~id
            u64 run = 0;
#pragma unroll 4
            for (uint32_t j = lane & 3; j < keep; j += 4) run += (uint32_t)order[j] > mine ? heavy[j] : 0;
            run += __shfl_xor_sync(kFull, run, 1);
            run += __shfl_xor_sync(kFull, run, 2);
            if (i < keep && (lane & 3) == 0 && run <= t && t < run + heavy[i])
                answer(row, ~mine, key_value((uint32_t)(order[i] >> 32)), total);
        }
        return true;
    }

    __device__ __forceinline__ u64 goal_of(uint32_t row, u64 total) const {
        const double x = (double)P.u[row] * (double)total;
        const u64 t = x > 0.0 ? (u64)x : 0;
        return t < total ? t : total - 1;
    }
    __device__ __forceinline__ void answer(uint32_t row, uint32_t id, float v, u64 total) const {
        P.ids[row] = (int32_t)id;
        if (P.logprob) P.logprob[row] = z_of(v, top, inv_t) - logf((float)total * 0x1p-40f);
    }
    // The running mass that the id drawn passes, worked out by one thread: 64-bit floating point is slow here.
    __device__ __forceinline__ u64 goal_for_all(uint32_t row, u64 total) const {
        if (threadIdx.x == 0) S.goal = goal_of(row, total);
        __syncthreads();
        return S.goal;
    }
    // own: this thread's kept mass.
    __device__ __forceinline__ void draw(uint32_t row, u64 own, u64 t, u64 total, u64 before, u64 mine, u64 least) const {
        locate([&](uint32_t i, float v) { return kept(i, v, least); }, own, t, before, mine,
               [&](uint32_t i) { answer(row, first + i, logit(i), total); });
        sync();   // no CTA ends while another may read its shared memory
    }
};

// The CTA's logits to shared memory one at a time, from group `whole` on, and -infinity to the last group's end; the
// largest of this thread's, NaN aside.
template <bool kHalf, int kThreads, bool kTeam, bool kCut>
__device__ __forceinline__ float load_tail(Sampler<kHalf, kThreads, kTeam, kCut> &A, uint4 *to, const uint8_t *l, uint32_t whole) {
    constexpr int kVec = kHalf ? 8 : 4, kSize = kHalf ? 2 : 4;
    float big = -INFINITY;
    const uint32_t end = (A.count + kVec - 1) / kVec * kVec;
#pragma unroll 4
    for (uint32_t i = whole * kVec + threadIdx.x; i < end; i += kThreads) {
        uint32_t b = kSize == 4 || A.P.type == BPE_BF16 ? 0xFF800000u : 0xFC00FC00u;   // -infinity
        if (kSize == 2 && A.P.type == BPE_BF16) b >>= 16;
        if (i < A.count) b = kHalf ? ((const unsigned short *)l)[i] : ((const uint32_t *)l)[i];
        if (kHalf)
            ((unsigned short *)to)[i] = (unsigned short)b;
        else
            ((uint32_t *)to)[i] = b;
        big = fmaxf(big, kHalf ? A.decode(b & 0xFFFFu) : __uint_as_float(b));
    }
    return big;
}

// The same, 16 bytes at a time where rows start on 16 bytes.
template <bool kHalf, int kThreads, bool kTeam, bool kCut>
__device__ __forceinline__ float load_row(Sampler<kHalf, kThreads, kTeam, kCut> &A, uint4 *to, const uint8_t *l, bool wide) {
    constexpr int kVec = kHalf ? 8 : 4;
    float big = -INFINITY;
    const uint32_t whole = wide ? A.count / kVec : 0;
#pragma unroll 8
    for (uint32_t g = threadIdx.x; g < whole; g += kThreads) {
        const uint4 q = __ldcs((const uint4 *)l + g);
        float v[kVec];
        A.unpack(q, v);
#pragma unroll
        for (int j = 0; j < kVec; j++) big = fmaxf(big, v[j]);
        to[g] = q;
    }
    return fmaxf(big, load_tail(A, to, l, whole));
}
// One row, whose logits are in place; big: the largest of those that this thread has seen.
template <bool kHalf, int kThreads, bool kTeam, bool kCut>
__device__ __forceinline__ void sample_row(Sampler<kHalf, kThreads, kTeam, kCut> &A, uint32_t row, float big, uint4 *to) {
    auto &S = A.S;
    const SampleParams &P = A.P;
    const uint32_t rank = A.rank, first = A.first, count = A.count;
    const uint32_t kmax = A.max_row(key_of(big));
    if (kmax == kKeyNegInf) {
        if (rank == 0 && threadIdx.x == 0) {
            P.ids[row] = -1;
            if (P.logprob) P.logprob[row] = -INFINITY;
        }
        A.sync();
        return;
    }
    A.top = key_value(kmax);
    if (A.top == INFINITY) {   // only infinities can be drawn: 0 in their place, -infinity elsewhere
        A.each([&](uint32_t i, float v) {
            const bool in = v == INFINITY;
            if (kHalf)
                ((unsigned short *)to)[i] = in ? 0 : P.type == BPE_BF16 ? 0xFF80 : 0xFC00;
            else
                ((float *)to)[i] = in ? 0.0f : -INFINITY;
        });
        __syncthreads();
        A.top = 0.0f;
    }
    const float temp = A.temp = P.f.d_temperature ? P.f.d_temperature[row] : P.f.temperature;
    if (!(temp >= kMinScale)) {   // the lowest id of the largest logit
        uint32_t low = 0;
        A.each([&](uint32_t i, float v) {
            if (v == A.top && i < count) low = max(low, ~(first + i));
        });
        low = A.max_row(low);
        if (rank == 0 && threadIdx.x == 0) {
            P.ids[row] = (int32_t)~low;
            if (P.logprob) P.logprob[row] = 0.0f;
        }
        A.sync();
        return;
    }
    const int32_t k = P.f.d_top_k ? P.f.d_top_k[row] : P.f.top_k;
    const float p = P.f.d_top_p ? P.f.d_top_p[row] : P.f.top_p;
    const float q = P.f.d_min_p ? P.f.d_min_p[row] : P.f.min_p;
    const u64 least = q > 0.0f ? (u64)(fminf(q, 1.0f) * kOne) : 0;
    A.inv_t = 1.0f / temp;
    const bool by_count = kCut && k >= 1 && (uint32_t)k < P.n_tok;
    if constexpr (kCut) {
        if (by_count && k <= kSmallK && A.small_list((uint32_t)k, p, least, row)) return;
    }
    if (threadIdx.x == 0) S.cut_v = -INFINITY, S.cut_idx = ~0u;   // keep all
    u64 total = 0, mine = 0, before, own;
    bool summed = false;
    if constexpr (kCut) {
        if (by_count) {
            A.template select<false, true>((u64)k, -1.0);
            if (p < 1.0f) {
                __syncthreads();
                A.read_cut();
                const u64 kept = A.sum_row(A.mass(0));
                if (threadIdx.x == 0) {
                    const double x = (double)p * (double)kept;
                    S.goal = x > 1.0 ? (u64)x : 1;
                }
                A.sync();   // the lists have been read by all, too
                A.template select<true, false>(S.goal, -1.0);
            }
        } else if (p < 1.0f) {
            summed = A.template select<true, true>(0, p > 0.0f ? (double)p : 0.0, &total, &mine) && !least;
        }
    }
    __syncthreads();
    A.read_cut();
    u64 t;
    if (summed && A.members() > 1) {   // the mass is known; only the CTA that holds the draw adds up its threads'
        A.sum_ctas(mine, before);
        t = A.goal_for_all(row, total);
        if (t >= before && t - before < mine) A.sum_cta(own = A.mass(0));
    } else {
        own = A.mass(least);
        mine = A.sum_cta(own);
        total = A.sum_ctas(mine, before);
        t = A.goal_for_all(row, total);
    }
    A.draw(row, own, t, total, before, mine, least);
}

template <bool kHalf, int kThreads, bool kTeam>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads)
k_sample(SampleParams P, uint32_t team, uint32_t slice, bool wide) {
    extern __shared__ __align__(16) uint8_t raw[];
    auto &S = *reinterpret_cast<SampleShared<kThreads, kTeam, true> *>(raw);
    const uint32_t row = kTeam ? blockIdx.x / team : blockIdx.x, rank = kTeam ? blockIdx.x % team : 0;
    const uint32_t first = min(P.n_tok, rank * slice), count = min(P.n_tok, first + slice) - first;
    // every CTA of the row has begun before another writes to its shared memory
    if (kTeam) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    Sampler<kHalf, kThreads, kTeam, true> A{S, P, S.row, rank, team, first, count};
    A.begin_row();
    const float big = load_row(A, S.row, (const uint8_t *)P.logits + (row * P.stride + first) * (kHalf ? 2 : 4), wide);
    if (kTeam) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    sample_row(A, row, big, S.row);
}

// Many rows of a small vocabulary, without top-k and top-p: each CTA takes rows in turn, and the next one's logits
// arrive while it draws from this one's.
template <bool kHalf, int kThreads>
__global__ void __launch_bounds__(kThreads, kRowCtas)
k_sample_rows(SampleParams P, uint32_t n_rows, uint32_t slice, bool wide) {
    extern __shared__ __align__(16) uint8_t raw[];
    auto &S = *reinterpret_cast<SampleShared<kThreads, false, false> *>(raw);
    constexpr int kVec = kHalf ? 8 : 4;
    const uint32_t groups = (P.n_tok + kVec - 1) / kVec, whole = wide ? P.n_tok / kVec : 0;
    Sampler<kHalf, kThreads, false, false> A{S, P, S.row, 0, 1, 0, P.n_tok};
    auto fetch = [&](uint32_t row, uint4 *to) {
        const uint8_t *l = (const uint8_t *)P.logits + row * P.stride * (kHalf ? 2 : 4);
        for (uint32_t g = threadIdx.x; g < whole; g += kThreads)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                         ::"r"((uint32_t)__cvta_generic_to_shared(to + g)), "l"(l + (uint64_t)g * 16) : "memory");
        asm volatile("cp.async.commit_group;" ::: "memory");
        if (whole < groups) load_tail(A, to, l, whole);
    };
    uint4 *now = S.row, *next = S.row + slice / kVec;
    if (blockIdx.x < n_rows) fetch(blockIdx.x, now);
    for (uint32_t row = blockIdx.x; row < n_rows; row += gridDim.x) {
        if (row + gridDim.x < n_rows) fetch(row + gridDim.x, next);
        A.data = now;
        A.begin_row();
        if (row + gridDim.x < n_rows)
            asm volatile("cp.async.wait_group 1;" ::: "memory");
        else
            asm volatile("cp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        float big = -INFINITY;
        for (uint32_t g = A.g0; g < A.g1; g++) big = fmaxf(big, A.most(now[g]));
        sample_row(A, row, big, now);
        __syncthreads();
        uint4 *t = now;
        now = next, next = t;
    }
}

// 0 for -infinity and NaN, and where z is none: an infinite distance times the 0 of an infinite temperature.
__device__ __forceinline__ u64 weight_of(float v, float top, float inv_t) {
    return v > -INFINITY ? weight(expf(fmaxf(z_of(v, top, inv_t), -31.75f))) : 0;
}

__device__ __forceinline__ u64 sum_all(u64 v, u64 *red) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    u64 t = 0;
    for (int i = 0; i < kSampThreads / 32; i++) t += red[i];
    return t;
}

// Vocabularies beyond a cluster's shared memory: one CTA per
// row reads it from L2 again in each step.  The kept tokens are those with a key above `cut`, and the
// first `ties` with the key `cut`; the cut is found bit by bit.
template <typename T>
__global__ void __launch_bounds__(kSampThreads) k_sample_stream(SampleParams P) {
    __shared__ u64 red[kSampThreads / 32];
    __shared__ u64 seg_mass[kSampThreads / 32];
    __shared__ uint32_t seg_ties[kSampThreads / 32];
    const uint64_t row = blockIdx.x;
    const T *l = (const T *)P.logits + row * P.stride;
    const uint32_t n = P.n_tok;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

    uint32_t kmax = kKeyNegInf;
    for (uint32_t i = threadIdx.x; i < n; i += kSampThreads) kmax = max(kmax, key_of(to_f32(l[i])));
    kmax = __reduce_max_sync(kFull, kmax);
    if (lane == 0) seg_ties[warp] = kmax;
    __syncthreads();
    for (int i = 0; i < kSampThreads / 32; i++) kmax = max(kmax, seg_ties[i]);
    __syncthreads();
    if (kmax == kKeyNegInf) {
        if (threadIdx.x == 0) {
            P.ids[row] = -1;
            if (P.logprob) P.logprob[row] = __uint_as_float(0xFF800000u);
        }
        return;
    }
    const float top = key_value(kmax);
    const float temp = P.f.d_temperature ? P.f.d_temperature[row] : P.f.temperature;
    const int32_t k = P.f.d_top_k ? P.f.d_top_k[row] : P.f.top_k;
    const float p = P.f.d_top_p ? P.f.d_top_p[row] : P.f.top_p;
    const float q = P.f.d_min_p ? P.f.d_min_p[row] : P.f.min_p;
    const bool greedy = !(temp >= kMinScale);
    const float inv_t = greedy ? 1.0f : 1.0f / temp;

    uint32_t cut = 0, ties = 0;          // keep all
    const u64 least = q > 0.0f ? (u64)(fminf(q, 1.0f) * kOne) : 0;
    if (greedy) {
        cut = kmax;
        ties = 1;
    } else {
        if (k >= 1 && (uint32_t)k < n) {
            for (int bit = 31; bit >= 0; bit--) {
                const uint32_t c = cut | 1u << bit;
                u64 cnt = 0;
                for (uint32_t i = threadIdx.x; i < n; i += kSampThreads) cnt += key_of(to_f32(l[i])) >= c;
                if (sum_all(cnt, red) >= (u64)k) cut = c;
            }
            u64 above = 0;
            for (uint32_t i = threadIdx.x; i < n; i += kSampThreads) above += key_of(to_f32(l[i])) > cut;
            ties = (uint32_t)((u64)k - sum_all(above, red));
        }
        if (p < 1.0f) {
            u64 mass = 0;
            for (uint32_t i = threadIdx.x; i < n; i += kSampThreads) {
                const float v = to_f32(l[i]);
                if (key_of(v) > cut) mass += weight_of(v, top, inv_t);
            }
            mass = sum_all(mass, red) + (ties ? ties * weight_of(key_value(cut), top, inv_t) : 0);
            const double e = (double)p * (double)mass;
            u64 edge = e > 1.0 ? (u64)e : 1;
            uint32_t c2 = 0;
            for (int bit = 31; bit >= 0; bit--) {
                const uint32_t c = c2 | 1u << bit;
                u64 m = 0;
                for (uint32_t i = threadIdx.x; i < n; i += kSampThreads) {
                    const float v = to_f32(l[i]);
                    if (key_of(v) >= c) m += weight_of(v, top, inv_t);
                }
                if (sum_all(m, red) >= edge) c2 = c;
            }
            u64 above = 0;
            for (uint32_t i = threadIdx.x; i < n; i += kSampThreads) {
                const float v = to_f32(l[i]);
                if (key_of(v) > c2) above += weight_of(v, top, inv_t);
            }
            above = sum_all(above, red);
            const u64 w = weight_of(key_value(c2), top, inv_t);
            const uint32_t t2 = (uint32_t)((edge - above + w - 1) / w);
            if (c2 > cut) cut = c2, ties = t2;
            else if (c2 == cut) ties = min(ties, t2);
        }
    }

    // each warp takes a contiguous segment; mass above the cut and ties in it
    const uint32_t seg = ((n + kSampThreads / 32 - 1) / (kSampThreads / 32) + 31) & ~31u;
    const uint32_t s0 = min(n, warp * seg), s1 = min(n, s0 + seg);
    u64 mass = 0;
    uint32_t eq = 0;
    for (uint32_t i = s0 + lane; i < s1; i += 32) {
        const float v = to_f32(l[i]);
        const uint32_t key = key_of(v);
        const u64 w = key >= cut ? weight_of(v, top, inv_t) : 0;
        if (key > cut && w >= least) mass += w;
        eq += key == cut;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mass += __shfl_xor_sync(kFull, mass, d);
    eq = __reduce_add_sync(kFull, eq);
    if (lane == 0) seg_mass[warp] = mass, seg_ties[warp] = eq;
    __syncthreads();
    u64 wc = ties ? weight_of(key_value(cut), top, inv_t) : 0;
    if (wc < least) wc = 0;
    u64 total = 0;
    uint32_t seen = 0;
    for (int i = 0; i < kSampThreads / 32; i++) total += seg_mass[i], seen += seg_ties[i];
    total += min(seen, ties) * wc;
    const float u = P.u[row];
    const double at = (double)u * (double)total;
    u64 t = at > 0.0 ? (u64)at : 0;
    if (t > total - 1) t = total - 1;
    // the warp whose segment holds it
    u64 before = 0;
    uint32_t eq_before = 0;
    for (int i = 0; i < warp; i++) before += seg_mass[i], eq_before += seg_ties[i];
    const u64 lo = before + min(eq_before, ties) * wc;
    const u64 hi = before + mass + min(eq_before + eq, ties) * wc;
    if (t < lo || t >= hi) return;
    for (uint32_t i0 = s0; i0 < s1; i0 += 32) {
        const uint32_t i = i0 + lane;
        const float v = i < s1 ? to_f32(l[i]) : 0.0f;
        const uint32_t key = i < s1 ? key_of(v) : 0;
        const u64 w = i < s1 && key >= cut ? weight_of(v, top, inv_t) : 0;
        u64 run = i < s1 && key > cut && w >= least ? w : 0;
        const unsigned tie = __ballot_sync(kFull, i < s1 && key == cut);
        const uint32_t rank = eq_before + __popc(tie & (0xFFFFFFFFu >> (31 - lane)));
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const u64 o = __shfl_up_sync(kFull, run, d);
            if (lane >= d) run += o;
        }
        const unsigned past = __ballot_sync(kFull, before + run + min(rank, ties) * wc > t);
        if (past) {
            if (lane == __ffs(past) - 1) {
                P.ids[row] = (int32_t)i;
                if (P.logprob)
                    P.logprob[row] = greedy ? 0.0f : (float)((double)z_of(v, top, inv_t) - log((double)total * 0x1p-40));
            }
            return;
        }
        before += __shfl_sync(kFull, run, 31);
        eq_before += __popc(tie);
    }
}

template <bool kHalf, int kThreads, bool kTeam>
int launch_team(bpe_ctx *ctx, const SampleParams &P, uint32_t n_rows, uint32_t team, uint32_t slice, bool wide) {
    auto k = k_sample<kHalf, kThreads, kTeam>;
    static std::atomic<uint64_t> devices{0};
    BPE_CUDA(ctx, allow_shared(k, ctx->device, kMaxShared, devices), "head_sample");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n_rows * team);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(SampleShared<kThreads, kTeam, true>) + (size_t)slice * (kHalf ? 2 : 4);
    cfg.stream = ctx->stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {team, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = kTeam ? 1 : 0;
    BPE_CUDA(ctx, cudaLaunchKernelEx(&cfg, k, P, team, slice, wide), "head_sample launch");
    return BPE_OK;
}

template <bool kHalf, int kThreads>
int launch_rows(bpe_ctx *ctx, const SampleParams &P, uint32_t n_rows, uint32_t slice, bool wide) {
    auto k = k_sample_rows<kHalf, kThreads>;
    static std::atomic<uint64_t> devices{0};
    BPE_CUDA(ctx, allow_shared(k, ctx->device, kMaxShared, devices), "head_sample");
    const size_t smem = sizeof(SampleShared<kThreads, false, false>) + 2 * (size_t)slice * (kHalf ? 2 : 4);
    const uint32_t fit = (uint32_t)(kSmShared / (smem + 1024)), most = kRowCtas, per_sm = fit < most ? fit : most;
    const uint32_t grid = per_sm * (uint32_t)ctx->sm_count;
    k<<<n_rows < grid ? n_rows : grid, kThreads, smem, ctx->stream>>>(P, n_rows, slice, wide);
    BPE_CUDA(ctx, cudaGetLastError(), "head_sample launch");
    return BPE_OK;
}

template <bool kHalf>
int launch(bpe_ctx *ctx, const SampleParams &P, uint32_t n_rows) {
    constexpr uint32_t kSize = kHalf ? 2 : 4, kVec = 16 / kSize;
    constexpr uint32_t kMost = (uint32_t)((kMaxShared - sizeof(SampleShared<1024, true, true>)) / 16) * kVec;   // tokens of a CTA
    static_assert(kMost <= 1024 * 104, "tokens of a thread");
    if (P.n_tok > kMaxTeam * kMost || n_rows > 0x0FFFFFFFu) {
        auto k = P.type == BPE_F32 ? k_sample_stream<float>
                 : P.type == BPE_BF16 ? k_sample_stream<__nv_bfloat16> : k_sample_stream<__half>;
        k<<<n_rows, kSampThreads, 0, ctx->stream>>>(P);
        BPE_CUDA(ctx, cudaGetLastError(), "head_sample launch");
        return BPE_OK;
    }
    const bool wide = (uintptr_t)P.logits % 16 == 0 && (n_rows == 1 || P.stride % kVec == 0);
    uint32_t team = (P.n_tok + kMost - 1) / kMost;
    // A few rows without a small top-k, whose every logit needs an exponential: while SMs are idle, more CTAs a row
    // (1 x 32,256: 16 us with 8, 22 with 1); with a small top-k the barriers cost more (33 x 32,256: 18 us with 8, 14 with 1).
    const bool small_k = P.f.d_top_k || (P.f.top_k >= 1 && P.f.top_k <= kSmallK);
    while (!small_k && team * 2 <= kMaxTeam && (uint64_t)n_rows * team * 2 <= (uint64_t)ctx->sm_count && P.n_tok >= team * 2 * 4096) team *= 2;
    const uint32_t slice = ((P.n_tok + team - 1) / team + kVec - 1) / kVec * kVec;
    const bool by_cut = P.f.d_top_k || P.f.top_k >= 1 || P.f.d_top_p || P.f.top_p < 1.0f;   // many short steps
    // Where rows wait for an SM, small CTAs, so that several share one and cover each other's latency; else the
    // threads that finish a row soonest.  In us, with CTAs of 256 / 512 / 1024 threads: 1,548 x 15,500 bf16 top-p
    // 99 / 116 / 165; 256 x 32,256 bf16 top-p 47 / 41 / 46; 152 x 16,000 bf16 top-p 23 / 18 / 17.  Rows without a cut of
    // their own by k_sample_rows: 4,096 x 4,352 bf16 25 against 39 with 256 threads a row; with one, its steps of few
    // threads take longer (2,060 x 2,902 f32 top-k: 64 against 47).  In clusters, 512 threads where two CTAs fit an SM,
    // since clusters of whole SMs do not fill the GPU: 38 x 65,536 f32 top-p 25 / 36 with 512 / 1024, and 4 x 100,000
    // 21 / 23; longer slices want the threads (152 x 70,000 f32 top-p 65 / 62).
    const bool many = (uint64_t)n_rows * team > (uint64_t)ctx->sm_count;
    if (team > 1)
        return slice * kSize <= 80 * 1024 ? launch_team<kHalf, 512, true>(ctx, P, n_rows, team, slice, wide)
                                          : launch_team<kHalf, 1024, true>(ctx, P, n_rows, team, slice, wide);
    if (slice <= 5120 && n_rows > 4 * (uint32_t)ctx->sm_count && !by_cut) return launch_rows<kHalf, 128>(ctx, P, n_rows, slice, wide);
    if (n_rows > 2 * (uint32_t)ctx->sm_count && slice * kSize <= 39 * 1024)
        return launch_team<kHalf, 256, false>(ctx, P, n_rows, 1, slice, wide);
    if (slice <= 8192 || (many && slice * kSize <= 80 * 1024))
        return launch_team<kHalf, 512, false>(ctx, P, n_rows, 1, slice, wide);
    return launch_team<kHalf, 1024, false>(ctx, P, n_rows, 1, slice, wide);
}

}  // namespace
}  // namespace bpe

using namespace bpe;

extern "C" int head_sample(bpe_ctx *ctx, const void *d_logits, uint64_t stride, int type, uint32_t n_rows, uint32_t n_tok,
                           const float *d_u, const head_filters *filters, int32_t *d_ids_out, float *d_logprob_out) {
    if (!ctx) return BPE_ERR_INVALID_ARG;
    if (!head_type_ok(type)) return fail(ctx, BPE_ERR_INVALID_ARG, "head_sample: unknown element type");
    if (n_tok == 0 || n_tok > BPE_HEAD_MAX_TOKENS)
        return fail(ctx, BPE_ERR_INVALID_ARG, "head_sample: %u tokens outside 1..%u", n_tok, BPE_HEAD_MAX_TOKENS);
    if (n_rows == 0) return BPE_OK;
    if (n_rows > 0x7FFFFFFFu) return fail(ctx, BPE_ERR_INVALID_ARG, "head_sample: %u rows", n_rows);
    if (!d_logits || !d_u || !d_ids_out) return fail(ctx, BPE_ERR_INVALID_ARG, "head_sample: null pointer");
    if (n_rows > 1 && stride < n_tok) return fail(ctx, BPE_ERR_INVALID_ARG, "head_sample: the row stride is below n_tok");
    if (const int rc = head_report(ctx)) return rc;
    BPE_CUDA(ctx, cudaSetDevice(ctx->device), "cudaSetDevice");
    const head_filters none{1.0f, 0, 1.0f, 0.0f, nullptr, nullptr, nullptr, nullptr};
    SampleParams P{d_logits, stride, n_tok, type, d_u, filters ? *filters : none, d_ids_out, d_logprob_out};
    return type == BPE_F32 ? launch<false>(ctx, P, n_rows) : launch<true>(ctx, P, n_rows);
}
