// head_row.cuh -- a row of logits as the scoring and training kernels of the
// output head see it (head_score.cu, head_distill.cuh): its vectors of 16 bytes,
// its softmax, and the sums over its threads and CTAs.
//
// A row of V logits is read once, by a warp, a CTA or a cluster.  Its bytes, V x 2
// or 4, are the floor; what competes with them is issue slots.  A logit of 16 bits
// takes about six instructions (a share of two copies, raise, largest, unpack, half
// a fused step, an exponential, one or two half additions), and 130 to 190 a thread
// for each row come on top, so that many rows have few threads each.  With the
// loads two tiles ahead, 8,192 x 32,256 bf16 are summed in 81 us (6.5 TB/s, 97% of
// the copy rate), 8,192 x 1,000 in 7 (2.3 TB/s).
#pragma once

#include "device.cuh"
#include "head.cuh"
#include "internal.h"

namespace bpe {

typedef unsigned long long u64;

constexpr int kMaxTeam = 8;                // CTAs of a row: a cluster
constexpr int kMost = 256;                 // threads of a row in a CTA of a cluster
constexpr int kMostWarps = 16;             // of any CTA
// A row's threads, kLanes: a warp of a CTA that takes eight rows, or a CTA of 64, 128, 256 or 512.
constexpr int kWarpRows = 8;

struct RowParams {
    const void *logits;
    uint64_t stride;
    uint32_t n_tok;
    float temperature;
    const float *d_temperature;

    // c = 1 / temperature, or infinity for the limit
    __device__ __forceinline__ float inverse(uint32_t row) const {
        const float t = d_temperature ? d_temperature[row] : temperature;
        return t >= kMinScale ? 1.0f / t : INFINITY;
    }
};

// ------------------------------------------------------------ elements ---
template <typename T> struct Bits;
template <> struct Bits<float> { static constexpr uint32_t kNegInf = 0xFF800000u, kShift = 0; };
template <> struct Bits<__nv_bfloat16> { static constexpr uint32_t kNegInf = 0xFF80FF80u, kShift = 16; };
template <> struct Bits<__half> { static constexpr uint32_t kNegInf = 0xFC00FC00u, kShift = 13; };   // of 32 bits, the low ones that carry nothing

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

__device__ __forceinline__ void unpack(const uint4 &q, float (&v)[4], float) {
    v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void unpack(const uint4 &q, float (&v)[8], __nv_bfloat16) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; i++) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack(const uint4 &q, float (&v)[8], __half) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 f = __half22float2(*(const __half2 *)&w[i]);
        v[2 * i] = f.x, v[2 * i + 1] = f.y;
    }
}

// A row that starts anywhere, as the aligned vectors of 16 bytes that hold it.  Element e of vector i is token
// i * kVec + e - shift; the first and the last vector may reach beyond the row, which is neither read nor written there.
template <typename T> struct RowView {
    static constexpr uint32_t kVec = 16 / sizeof(T);
    T *at;              // the vector in which the row starts
    uint32_t shift;     // elements of it before the row
    uint32_t end;       // shift + tokens

    __device__ __forceinline__ RowView(const void *base, uint64_t stride, uint32_t row, uint32_t n) {
        T *const p = (T *)base + row * stride;
        shift = (uint32_t)((uintptr_t)p & 15) / sizeof(T);
        at = p - shift;     // a pointer rounded as a number would be one to any memory, whose stores are slower
        end = shift + n;
    }
    __device__ __forceinline__ uint32_t vecs() const { return (end + kVec - 1) / kVec; }
    __device__ __forceinline__ bool whole(uint32_t i) const { return i * kVec >= shift && (i + 1) * kVec <= end; }
    // vector i, -infinity where it reaches beyond the row
    __device__ __forceinline__ uint4 load(uint32_t i) const {
        return whole(i) ? *((const uint4 *)at + i) : edge(*this, i);
    }
    static __device__ __noinline__ uint4 edge(RowView r, uint32_t i) {
        uint4 q = make_uint4(Bits<T>::kNegInf, Bits<T>::kNegInf, Bits<T>::kNegInf, Bits<T>::kNegInf);
#pragma unroll
        for (uint32_t e = 0; e < kVec; e++) {
            const uint32_t p = i * kVec + e;
            if (p >= r.shift && p < r.end) put(q, e, r.at[p]);
        }
        return q;
    }
    static __device__ __forceinline__ void put(uint4 &q, uint32_t e, T v) {
        uint32_t *w = (uint32_t *)&q;
        if (sizeof(T) == 4) {
            w[e] = *(const uint32_t *)&v;
        } else {
            const uint32_t b = *(const unsigned short *)&v;
            w[e / 2] = e & 1 ? (w[e / 2] & 0xFFFFu) | b << 16 : (w[e / 2] & 0xFFFF0000u) | b;
        }
    }
};

// Vector i of a gradient, in the place of the row's.  What is not a whole vector, or starts elsewhere in one than the row
// does, goes element by element, in a function of its own: written out here, its stores take issue slots when they do not
// run.  `direct`: known to be neither.
template <typename T> __device__ __noinline__ void put_elements(RowView<T> out, RowView<T> row, uint32_t i, uint4 q) {
    const T *const v = (const T *)&q;
    constexpr uint32_t kVec = RowView<T>::kVec;
#pragma unroll
    for (uint32_t e = 0; e < kVec; e++) {
        const uint32_t at = i * kVec + e;
        if (at >= row.shift && at < row.end) out.at[out.shift + at - row.shift] = v[e];
    }
}
template <typename T>
__device__ __forceinline__ void put_vector(const RowView<T> &out, const RowView<T> &row, uint32_t i, const float (&v)[RowView<T>::kVec], bool direct) {
    const uint4 q = pack16(v, T());
    if (direct || (out.shift == row.shift && row.whole(i))) *((uint4 *)out.at + i) = q;
    else put_elements(out, row, i, q);
}

// Whether any row starts inside a vector.
template <typename T> inline bool row_shifts(const void *base, uint64_t stride, uint32_t n_rows) {
    return (uintptr_t)base % 16 || (n_rows > 1 && stride * sizeof(T) % 16);
}

// ------------------------------------------------------------ softmax ---
// z of a logit, for every m and c (NaN counts as -infinity).
__device__ __forceinline__ float z_any(float v, float m, float c) {
    const float d = v - m;
    return v == m ? 0.0f : d > -INFINITY ? d * c : -INFINITY;   // a NaN compares false
}

// ------------------------------------------------------- the usual row ---
// Sums over rows are taken in one pass: every thread keeps the largest logit that it has met, and its sums relative to
// that one, which are scaled when a larger one comes.  In powers of two, z = v (c log2 e) - R with R = m (c log2 e) rounded
// once, so that a logit costs one fused step and one exponential.
//
// That needs numbers that stay finite: logits below `kLow` count as it, and what comes out holds where they have no weight,
// and where the largest logit's own z, what R was rounded by, is at most one step of the exponent: where the row is `usual`.
// Others (masked by the type's lowest value or another far from 0 throughout, infinite, at far temperatures, |m| / T above
// 2^24) take the general form, softmax_any.
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

constexpr float kMostMc = 0x1p24f;         // m c log2 e below 2^24.6: numbers are 2 apart there

template <typename T> struct Usual {
    static constexpr float kLow = -0x1p60f, kLeast = -0x1p50f, kMost = 0x1p50f, kMinC = 0x1p-40f, kMaxC = 0x1p20f;
};
template <> struct Usual<__half> {   // its lowest number is -65,504; from -16,384 down by 2^-6 a unit e^-768 is left of it
    static constexpr float kLow = -65504.0f, kLeast = -16384.0f, kMost = 65504.0f, kMinC = 0x1p-6f, kMaxC = 0x1p20f;
};
template <typename T> __device__ __forceinline__ bool usual(float m, float c) {
    float mc;   // written out: as an expression among the others it gives distillation with gradient another order of instructions
    asm("mul.rn.f32 %0, %1, %2;" : "=f"(mc) : "f"(fabsf(m)), "f"(c));   // (8,192 x 32,256 bf16: 173.9 us, 171.4 so)
    return m >= Usual<T>::kLeast && m <= Usual<T>::kMost && c >= Usual<T>::kMinC && c <= Usual<T>::kMaxC && mc <= kMostMc;
}
// What the sums run with in its place until that is known (a far c would make them NaN; they are not used then).
template <typename T> __device__ __forceinline__ float usual_c(float c) {
    return c >= Usual<T>::kMinC && c <= Usual<T>::kMaxC ? c : 1.0f;
}

__device__ __forceinline__ float exp2_of(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// R of a largest logit m, but no less than -2^25, which is below any usual row's.  Far from 0 the rounding of m c2 is more than a
// step of the exponent, from 2^31 on more than all of its range, so that what a tile, a warp or a CTA of masked logits alone
// weighs relative to its own largest may come out infinite.  Relative to -2^25 it is 0, as it is beside the row's largest.
__device__ __forceinline__ float base_of(float m, float c2) { return fmaxf(__fmul_rn(m, c2), -0x1p25f); }

// Two numbers of 32 bits in one register pair.
struct Pair {
    u64 b;
    Pair() = default;
    __device__ __forceinline__ Pair(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(x), "f"(y)); }
    __device__ __forceinline__ float2 both() const {
        float2 f;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(b));
        return f;
    }
};
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.b) : "l"(a.b), "l"(b.b), "l"(c.b));
    return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
    return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(a.b), "l"(b.b));
    return r;
}

// Logits by words of 32 bits: raised to kLow (a NaN too), the larger of two, the largest of a word.
template <typename T> struct Words;
template <> struct Words<float> {
    using W = float;
    static __device__ __forceinline__ W low() { return Usual<float>::kLow; }
    static __device__ __forceinline__ W larger(W a, W b) { return fmaxf(a, b); }
    static __device__ __forceinline__ float largest(W a) { return a; }
};
template <> struct Words<__nv_bfloat16> {
    using W = __nv_bfloat162;
    static __device__ __forceinline__ W low() { return __float2bfloat162_rn(Usual<__nv_bfloat16>::kLow); }
    static __device__ __forceinline__ W larger(W a, W b) { return __hmax2(a, b); }
    static __device__ __forceinline__ float largest(W a) { return fmaxf(__low2float(a), __high2float(a)); }
};
template <> struct Words<__half> {
    using W = __half2;
    static __device__ __forceinline__ W low() { return __float2half2_rn(Usual<__half>::kLow); }
    static __device__ __forceinline__ W larger(W a, W b) { return __hmax2(a, b); }
    static __device__ __forceinline__ float largest(W a) { return fmaxf(__low2float(a), __high2float(a)); }
};
// Raises a vector, and gives the word of its largest logits.
template <typename T> __device__ __forceinline__ typename Words<T>::W raise(uint4 &q) {
    using F = Words<T>;
    typename F::W *w = (typename F::W *)&q;
#pragma unroll
    for (int e = 0; e < 4; e++) w[e] = F::larger(w[e], F::low());
    return F::larger(F::larger(w[0], w[1]), F::larger(w[2], w[3]));
}

template <int kLanes> __device__ __forceinline__ uint32_t row_thread() { return kLanes == 32 ? threadIdx.x & 31 : threadIdx.x; }

// kSize vectors a thread, of the CTA's share of a row.
template <typename T, int kSize, int kLanes> struct Tile {
    static constexpr uint32_t kVecs = kSize * kLanes;
    uint4 q[kSize];

    // Raises the tile; gives its largest logit.
    __device__ __forceinline__ float raise_all() {
        typename Words<T>::W m = raise<T>(q[0]);
#pragma unroll
        for (int u = 1; u < kSize; u++) m = Words<T>::larger(m, raise<T>(q[u]));
        return Words<T>::largest(m);
    }
    __device__ __forceinline__ static uint32_t place(uint32_t i0, int u) { return i0 + u * kLanes + row_thread<kLanes>(); }
    // No vector from i0 on ends outside the row or the share.
    __device__ __forceinline__ static bool inside(const RowView<T> &row, uint32_t i0, uint32_t hi) {
        return (i0 > 0 || row.shift == 0) && i0 + kVecs <= min(hi, row.end / RowView<T>::kVec);
    }
    __device__ __forceinline__ static uint4 fill() {
        return make_uint4(Bits<T>::kNegInf, Bits<T>::kNegInf, Bits<T>::kNegInf, Bits<T>::kNegInf);
    }
};

// The CTA's share of a row on its way through shared memory, kAhead tiles ahead of where it is read.  Every thread copies
// (asynchronously, without registers) what it will read itself, so that no barrier is needed.  A share that is kept has a
// slot for every tile, and stays for a second look.
template <typename T, int kSize, int kLanes> struct Feed {
    using Tiles = Tile<T, kSize, kLanes>;
    static constexpr int kAhead = 2;
    static constexpr uint32_t kBytes = Tiles::kVecs * 16, kStep = kLanes * 16;   // of a tile, from a thread's vector to its next
    RowView<T> row;
    const char *from;          // this thread's first vector
    uint32_t mine;             // its place in the first slot, an address of 32 bits
    uint32_t lo, hi;
    bool kept;

    __device__ __forceinline__ Feed(const RowView<T> &r, void *shared, uint32_t lo_, uint32_t hi_, bool kept_ = false, bool reads = true)
        : row(r), from((const char *)r.at + (uint64_t)(lo_ + row_thread<kLanes>()) * 16),
          mine((uint32_t)__cvta_generic_to_shared(shared) + row_thread<kLanes>() * 16), lo(lo_), hi(hi_), kept(kept_) {
        if (reads) start();
    }
    __device__ __forceinline__ void start() const {
#pragma unroll
        for (int n = 0; n < kAhead; n++) ask(n);
    }
    __device__ __forceinline__ uint32_t slot(uint32_t n) const { return mine + (kept ? n : n % kAhead) * kBytes; }
    static __device__ __forceinline__ void copy(uint32_t to, const void *from) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    }
    __device__ __forceinline__ uint32_t steps() const { return (hi - lo + Tiles::kVecs - 1) / Tiles::kVecs; }
    // tile n's copies, as one group (an empty one behind the share)
    __device__ __forceinline__ void ask(uint32_t n) const {
        const uint32_t i0 = lo + n * Tiles::kVecs;
        if (Tiles::inside(row, i0, hi)) {
            const uint32_t to = slot(n);
            const char *const f = from + (uint64_t)n * kBytes;
#pragma unroll
            for (int u = 0; u < kSize; u++) copy(to + u * kStep, f + u * kStep);
        } else if (i0 < hi) {
            ask_edge(i0, slot(n));
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ void ask_edge(uint32_t i0, uint32_t to) const {
#pragma unroll 1
        for (uint32_t i = i0 + row_thread<kLanes>(); i < i0 + Tiles::kVecs; i += kLanes, to += kStep) {
            if (i < hi && row.whole(i)) {
                copy(to, (const uint4 *)row.at + i);
                continue;
            }
            const uint4 q = i < hi ? row.load(i) : Tiles::fill();
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(q.x), "r"(q.y), "r"(q.z), "r"(q.w) : "memory");
        }
    }
    // tile n, in order; then the copies of the one that takes its slot
    __device__ __forceinline__ void next(Tiles &t, uint32_t n) const {
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
        again(t, n);
        ask(n + kAhead);
    }
    // a tile that is still there
    __device__ __forceinline__ void again(Tiles &t, uint32_t n) const {
        const uint32_t at = slot(n);
#pragma unroll
        for (int u = 0; u < kSize; u++)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(t.q[u].x), "=r"(t.q[u].y), "=r"(t.q[u].z), "=r"(t.q[u].w)
                         : "r"(at + u * kStep) : "memory");
    }
};

// A thread's sums, relative to 2^r: the largest logit of the warp's first tile, and a larger one only where that is 2^kSlack
// above it, which is rare.  Larger numbers lose nothing; but z counts from r too, and a sum of z that has a far larger one
// taken off its terms at the end would lose as much, so that entropies allow little.
template <typename T, bool kEntropy> struct Running {
    static constexpr float kSlack = kEntropy ? 4.0f : 64.0f;
    float most, r;      // the largest logit; what the sums are relative to
    Pair s, sz;

    __device__ __forceinline__ explicit Running(float c2) : most(Usual<T>::kLow), r(__fmul_rn(Usual<T>::kLow, c2)), s(0, 0), sz(0, 0) {}
    __device__ __forceinline__ void move(float to) {   // no less than r
        const float d = r - to, f = exp2_of(d);
        if (kEntropy) sz = mul2(fma2(s, Pair(d, d), sz), Pair(f, f));
        s = mul2(s, Pair(f, f));
        r = to;
    }
    // Before the first tile, whose largest logit is m.
    __device__ __forceinline__ void begin(float m, float c2) {
        r = base_of(key_value(__reduce_max_sync(kFull, key_of(m))), c2);
    }
    // Adds a raised tile whose largest logit is m.
    template <int kSize, int kLanes> __device__ __forceinline__ void add(const Tile<T, kSize, kLanes> &t, float m, float c2) {
        constexpr int kVec = RowView<T>::kVec;
        most = fmaxf(most, m);
        if (fmaf(m, c2, -r) > kSlack) move(__fmul_rn(m, c2));
        const Pair k(c2, c2), off(-r, -r);
#pragma unroll
        for (int u = 0; u < kSize; u++) {
            float v[kVec];
            unpack(t.q[u], v, T());
#pragma unroll
            for (int e = 0; e < kVec; e += 2) {
                const Pair z = fma2(Pair(v[e], v[e + 1]), k, off);
                const float2 x = z.both();
                const Pair w(exp2_of(x.x), exp2_of(x.y));
                s = add2(s, w);
                if (kEntropy) sz = fma2(w, z, sz);
            }
        }
    }
};

// ------------------------------------------------- sums over a row's CTAs ---
__device__ __forceinline__ uint32_t far_addr(const void *p, uint32_t rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ void far_store(float4 *p, uint32_t rank, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(far_addr(p, rank)), "f"(v.x), "f"(v.y), "f"(v.z),
                 "f"(v.w) : "memory");
}
__device__ __forceinline__ u64 far_load(const u64 *p, uint32_t rank) {
    u64 v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(far_addr(p, rank)) : "memory");
    return v;
}

struct TeamShared {
    float4 red[kMostWarps];
    float4 slot[2][kMaxTeam];
};

// The threads of a row: a warp, a CTA, or the CTAs of a cluster.
template <int kLanes, bool kTeam> struct Team {
    static_assert(kLanes <= 32 * kMostWarps && (!kTeam || kLanes == kMost), "clusters are of CTAs of kMost");
    static constexpr bool kWarp = kLanes == 32;
    static constexpr int kWarps = kLanes / 32;
    TeamShared &S;         // not there for a warp
    uint32_t rank, size, thread;
    int lane, warp, turn;  // a thread beyond kLanes is of a warp that helps

    __device__ __forceinline__ Team(TeamShared &s, uint32_t team)
        : S(s), rank(kTeam ? blockIdx.x % team : 0), size(kTeam ? team : 1), thread(row_thread<kLanes>()), lane(threadIdx.x & 31),
          warp(kWarp ? 0 : threadIdx.x >> 5), turn(0) {}

    __device__ __forceinline__ void sync_cta() const {   // or the warp
        if (kWarp) __syncwarp();
        else __syncthreads();
    }
    // A CTA's shared memory is there for the others once it runs, and until it ends: the first exchange comes after the one
    // barrier's wait, the end after the other's.  Neither orders memory.
    __device__ __forceinline__ void arrive() const {
        if (kTeam) {
            __syncwarp();
            asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
        }
    }
    __device__ __forceinline__ void wait() const {
        if (kTeam) {
            __syncwarp();
            asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        }
    }
    // One value of each CTA to all: S.slot[turn][r] is CTA r's.  The slots of one exchange are written again two exchanges
    // later, when a barrier has shown that all have read them.
    __device__ __forceinline__ void exchange(float4 v) {
        turn ^= 1;
        if (threadIdx.x < size) far_store(&S.slot[turn][rank], threadIdx.x, v);
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    // The warps' values combined in the order of warps and CTAs; every thread gets the result.
    template <typename F> __device__ __forceinline__ float4 across(float4 v, F f) {
        if (kWarp) return v;
        __syncthreads();
        if (lane == 0 && warp < kWarps) S.red[warp] = v;
        __syncthreads();
        v = S.red[0];
#pragma unroll
        for (int i = 1; i < kWarps; i++) v = f(v, S.red[i]);
        if (!kTeam) return v;
        exchange(v);
        v = S.slot[turn][0];
        for (uint32_t r = 1; r < size; r++) v = f(v, S.slot[turn][r]);
        return v;
    }
    __device__ __forceinline__ float max(float v) {   // of values that are not NaN
        v = key_value(__reduce_max_sync(kFull, key_of(v)));
        return across(make_float4(v, 0, 0, 0), [](float4 a, float4 b) { return make_float4(fmaxf(a.x, b.x), 0, 0, 0); }).x;
    }
    __device__ __forceinline__ float4 sum(float4 v) {
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
            v.x += __shfl_xor_sync(kFull, v.x, d), v.y += __shfl_xor_sync(kFull, v.y, d);
            v.z += __shfl_xor_sync(kFull, v.z, d), v.w += __shfl_xor_sync(kFull, v.w, d);
        }
        return across(v, [](float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); });
    }
};

// The largest logit, the sum of exp(z) and that of exp(z) z.
struct Softmax { float m, s, sz; };
struct SoftmaxAny { Softmax all; int turn; };

// Sums relative to the largest m c2 of kN lanes' out of each lane's own, added up.
template <bool kEntropy, int kN> __device__ __forceinline__ float4 join_lanes(float4 v, float c2) {
    float m = v.x;
#pragma unroll
    for (int d = kN / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, d));
    const float d = base_of(v.x, c2) - base_of(m, c2), f = exp2_of(d);
    v = make_float4(m, v.y * f, kEntropy ? fmaf(v.y, d, v.z) * f : 0.0f, v.w);
#pragma unroll
    for (int e = kN / 2; e > 0; e >>= 1) {
        v.y += __shfl_xor_sync(kFull, v.y, e);
        if (kEntropy) v.z += __shfl_xor_sync(kFull, v.z, e);
        v.w += __shfl_xor_sync(kFull, v.w, e);
    }
    return v;
}

// The threads' sums to the row's.  m is exact; s and sz count where the row is usual.  `count`, the first warp's, is added
// up over CTAs beside them.
template <typename T, bool kEntropy, int kLanes, bool kTeam>
__device__ __forceinline__ Softmax softmax_join(Team<kLanes, kTeam> &team, Running<T, kEntropy> a, float c2, float &count) {
    constexpr int kWarps = kLanes / 32;
    const float m = key_value(__reduce_max_sync(kFull, key_of(a.most)));
    a.move(base_of(m, c2));
    const float2 s = a.s.both(), sz = a.sz.both();
    float4 v = make_float4(m, s.x + s.y, sz.x + sz.y, team.warp == 0 ? count : 0.0f);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        v.y += __shfl_xor_sync(kFull, v.y, d);
        if (kEntropy) v.z += __shfl_xor_sync(kFull, v.z, d);
    }
    if (kLanes > 32) {
        if (team.lane == 0 && team.warp < kWarps) team.S.red[team.warp] = v;
        __syncthreads();
        v = join_lanes<kEntropy, kWarps>(team.S.red[team.lane % kWarps], c2);
    }
    if (kTeam) {
        team.wait();   // the others run
        team.exchange(v);
        const uint32_t o = team.lane % kMaxTeam;
        v = o < team.size ? team.S.slot[team.turn][o] : make_float4(Usual<T>::kLow, 0, 0, 0);
        v = join_lanes<kEntropy, kMaxTeam>(v, c2);
    }
    count = v.w;
    // relative to m itself rather than to m c2 rounded
    const float d = fmaf(v.x, c2, -__fmul_rn(v.x, c2)), f = exp2_of(-d);
    return {v.x, v.y * f, (v.z - d * v.y) * f * kLn2};
}

// Both in their general form: any logits and any c, two passes.  `load(i)` gives vector i; threads beyond the row's own add
// nothing.  (By value, and the team's turn given back: what a function that is called takes by reference lives in memory, in
// the usual rows' loops too.)
template <typename T, int kLanes, bool kTeam, typename L>
__device__ __noinline__ SoftmaxAny softmax_sums(Team<kLanes, kTeam> team, uint32_t lo, uint32_t hi, float c, L load) {
    constexpr int kVec = RowView<T>::kVec;
    if (team.thread >= (uint32_t)kLanes) lo = hi;
    float m = -INFINITY;
    for (uint32_t i = lo + team.thread; i < hi; i += kLanes) {
        float v[kVec];
        unpack(load(i), v, T());
#pragma unroll
        for (int e = 0; e < kVec; e++) m = fmaxf(m, v[e]);   // the other one where one is NaN
    }
    m = team.max(m);
    if (m == -INFINITY) return {{m, 0.0f, 0.0f}, team.turn};
    float s = 0, sz = 0;
    for (uint32_t i = lo + team.thread; i < hi; i += kLanes) {
        float v[kVec];
        unpack(load(i), v, T());
#pragma unroll
        for (int e = 0; e < kVec; e++) {
            const float z = z_any(v[e], m, c), x = expf(z);
            s += x;
            sz += x > 0.0f ? x * z : 0.0f;
        }
    }
    const float4 all = team.sum(make_float4(s, sz, 0, 0));
    return {{m, all.x, all.y}, team.turn};
}
template <typename T, int kLanes, bool kTeam, typename L>
__device__ __forceinline__ Softmax softmax_any(Team<kLanes, kTeam> &team, uint32_t lo, uint32_t hi, float c, L load) {
    const SoftmaxAny any = softmax_sums<T, kLanes, kTeam>(team, lo, hi, c, load);
    team.turn = any.turn;
    return any.all;
}

// Threads of a row, at least `least` of them.  A row of few threads takes longer, but loses less to what is done once for each
// thread and to barriers.  So it is for many rows, where the time of the last ones hardly counts: with `each` bytes of a warp's
// share for every warp beyond two an SM.  In us with 32 / 64 / 128 / 256 threads, bf16, 20 alternatives (each = 4): 8,192 rows
// of 1,000 17 / 25 / 40 / 70, 1,024 of 8,192 14 / 11 / 9.5 / 12.5, 256 of 8,192 14 / 9 / 6.8 / 6.5; without alternatives
// (each = 40), 32 / 256: 8,192 of 1,000 7 / 32, of 32,256 81 / 85, 1,024 of 8,192 5.1 / 5.9, 512 of 8,192 5.0 / 3.8.
inline int row_lanes(uint32_t n_rows, uint32_t bytes, uint32_t sms, int least, uint32_t each) {
    for (int lanes = least; lanes < kMost; lanes *= 2) {
        const uint64_t warps = (uint64_t)n_rows * (lanes / 32);
        if (warps > 2 * sms && (uint64_t)bytes * 32 / lanes <= each * (warps - 2 * sms)) return lanes;
    }
    return kMost;
}

// CTAs of a row, of 32 KB at least: more than one where there are too few rows for `each` CTAs an SM.  A cluster costs each of
// its CTAs some us, so that a split that no idle SM asks for is slower (333 x 250,000 f16, 64 alternatives: 52 / 59 / 72 us in
// 1 / 2 / 4; 1 x 32,256 f32 11 / 12 / 11).
inline uint32_t row_team(uint32_t n_rows, uint32_t bytes, uint32_t sms, uint32_t each) {
    uint32_t team = 1;
    while (team < (uint32_t)kMaxTeam && (uint64_t)n_rows * team * 2 <= (uint64_t)each * sms && bytes >= team * 2 * 32768u) team *= 2;
    return team;
}

// A kernel with `ctas` CTAs, or clusters of `team` of them.
template <typename K, typename P, typename... More>
inline int launch_rows(bpe_ctx *ctx, const char *what, K kernel, const P &params, uint32_t ctas, uint32_t team, int threads,
                       bool cluster, size_t shared, More... more) {
    if ((uint64_t)ctas * team > 0x7FFFFFFFu) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: too many rows", what);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas * team);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = ctx->stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {team, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 1 : 0;
    BPE_CUDA(ctx, cudaLaunchKernelEx(&cfg, kernel, params, team, more...), what);
    return BPE_OK;
}

}  // namespace bpe
