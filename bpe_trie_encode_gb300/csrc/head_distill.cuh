// head_distill.cuh -- divergence of rows of logits from a teacher's top
// alternatives, and its gradient in the same call.  head_distill.cu has the
// entry point; a file for each type compiles the kernels.
//
// The divergence needs the row's softmax and the logits of the listed tokens, which
// a warp of its own gathers while the others read the row.  Where the unlisted
// tokens are one class, their softmax is taken without the listed ones (a bit for
// each place of the row, in shared memory, says which), and the two are put together
// after: however little of the row the unlisted hold, their shares are exact, which
// a difference of sums is not.
//
// The gradient is g (Q p - q): all of it is written as if nothing were listed, then
// the listed tokens' places again.  A row up to 64 KB stays in shared memory between
// the sums and the writing; a longer one is read again from L2.  Bound by HBM, and by
// the latency between the two passes: 8,192 x 32,256 bf16, 64 listed: 88 us without
// the gradient, 168 with it (6.3 TB/s of reading and writing, 93% of the copy rate);
// 900 x 250,000 bf16 with the rest 73 us (6.2 TB/s); 400 x 250,000 f16 with the rest
// and the gradient 97 (4.1 TB/s).
//
// (Measured and slower: CTAs that stay and ask for the next row's tiles while they
// write this one's, 193 us for 8,192 x 32,256 against 169: its bookkeeping takes 28%
// more instructions.)
#pragma once

#include "head_row.cuh"

namespace bpe {

struct DistillParams {
    RowParams row;
    const int32_t *top_ids;
    const void *top_logprob;
    int top_type;
    uint32_t n_listed;
    int rest;
    float *loss;
    float grad;
    const float *d_grad;
    void *out;
    uint64_t out_stride;
};

// The launch, for each type of logits.
int distill_f32(bpe_ctx *ctx, const DistillParams &P, uint32_t n_rows);
int distill_bf16(bpe_ctx *ctx, const DistillParams &P, uint32_t n_rows);
int distill_f16(bpe_ctx *ctx, const DistillParams &P, uint32_t n_rows);

namespace {

constexpr int kEntries = (int)BPE_HEAD_MAX_TOP;   // alternatives that a teacher lists
constexpr uint32_t kMostShared = 200 * 1024, kSmShared = 228 * 1024;   // of a CTA, of an SM
constexpr uint32_t kKeep = 4;                     // tiles of a row that leave room for three CTAs on an SM

constexpr int kHash = 256;
// Threads of a CTA: a row's and a warp for the entries, or a warp for each of eight rows; and CTAs that fit an SM.
template <int kLanes> constexpr int kThreads = kLanes == 32 ? kWarpRows * 32 : kLanes + 32;
template <int kLanes> constexpr int kCtas = kLanes == 32 ? 3 : kLanes == 64 ? 9 : kLanes == 128 ? 5 : 3;

struct DistillShared {
    TeamShared team;
    uint32_t id[kEntries];            // ~0: none, or the same as one before
    float q[kEntries], v[kEntries];   // the token's q, of all its entries; its logit
    uint32_t hash[kHash];
    float q_sum, m, s;         // the sum of the entries' q; the listed tokens' softmax
    uint32_t twice;            // whether an id is listed twice
    uint32_t bits[1];          // a bit for each place of the CTA's vectors: listed
};

__device__ __forceinline__ float warp_max(float v) { return key_value(__reduce_max_sync(kFull, key_of(v))); }
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}

// x y, and 0 where x is 0 whatever y is.
__device__ __forceinline__ float product(float x, float y) { return x == 0.0f ? 0.0f : x * y; }

// q (log q - log p) - q + p = q (e^d - 1 - d), d = log p - log q, which is never below 0.  Where all q and all p add up to 1 the
// sum of these terms is the divergence, and one that is small, since teacher and student agree, is not the difference of far
// larger ones.
__device__ __forceinline__ float divergence(float q, float log_q, float log_p) {
    const float d = log_p - log_q;
    if (!(fabsf(d) < 1.0f)) return expf(log_p) - q - q * d;
    float r = 1.0f / 39916800;             // the exponential's series: e^d - 1 - d = d^2 (1/2! + d/3! + d^2/4! ...)
    r = fmaf(r, d, 1.0f / 3628800), r = fmaf(r, d, 1.0f / 362880), r = fmaf(r, d, 1.0f / 40320), r = fmaf(r, d, 1.0f / 5040);
    r = fmaf(r, d, 1.0f / 720), r = fmaf(r, d, 1.0f / 120), r = fmaf(r, d, 1.0f / 24), r = fmaf(r, d, 1.0f / 6), r = fmaf(r, d, 0.5f);
    return q * (d * d * r);
}

// The row's entries, four to a lane of the CTA's last warp, which deals with them while the others read the row.
struct Entries {
    static constexpr int kEach = kEntries / 32;
    uint32_t id[kEach];        // ~0: none
    float t[kEach], v[kEach];  // value, then log q; the token's logit

    template <typename T> __device__ __forceinline__ void load(const DistillParams &P, uint32_t r, const RowView<T> &row, int lane) {
#pragma unroll
        for (int j = 0; j < kEach; j++) {
            const uint32_t i = j * 32 + lane;
            id[j] = ~0u, t[j] = -INFINITY, v[j] = -INFINITY;
            if (i >= P.n_listed) continue;
            const uint64_t at = (uint64_t)r * P.n_listed + i;
            id[j] = (uint32_t)P.top_ids[at];
            t[j] = P.top_type == BPE_F32    ? ((const float *)P.top_logprob)[at]
                   : P.top_type == BPE_BF16 ? to_f32(((const __nv_bfloat16 *)P.top_logprob)[at])
                                            : to_f32(((const __half *)P.top_logprob)[at]);
        }
#pragma unroll
        for (int j = 0; j < kEach; j++) {
            if (id[j] >= P.row.n_tok || !(t[j] > -INFINITY)) id[j] = ~0u, t[j] = -INFINITY;
            if (id[j] != ~0u) v[j] = to_f32(row.at[row.shift + id[j]]);
        }
    }
    // q and the tokens to shared memory.  An id that comes twice is found by a table of hashes; then (hardly ever) every
    // entry looks all others through, so that the sums are in the order of entries.
    __device__ __forceinline__ void weigh(DistillShared &S, const DistillParams &P, float c, int lane) {
        float m = -INFINITY, sum = 0, log_s = 0;
        if (!P.rest) {         // the softmax of the listed values
#pragma unroll
            for (int j = 0; j < kEach; j++) m = fmaxf(m, t[j]);
            m = warp_max(m);
#pragma unroll
            for (int j = 0; j < kEach; j++) {
                t[j] = id[j] != ~0u ? z_any(t[j], m, 1.0f) : -INFINITY;
                sum += expf(t[j]);
            }
            log_s = logf(warp_sum(sum));
        }
        float q_sum = 0;
        bool twice = false;
#pragma unroll
        for (int j = 0; j < kHash / 32; j++) S.hash[j * 32 + lane] = ~0u;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < kEach; j++) {
            const uint32_t i = j * 32 + lane;
            if (t[j] > -INFINITY) t[j] -= log_s;
            const float q = expf(t[j]);
            q_sum += q;
            S.id[i] = id[j], S.q[i] = q, S.v[i] = v[j];
            if (id[j] == ~0u) continue;
            // at most 128 of 256 places are taken; ids at equal distances are spread as others are
            for (uint32_t h = fmix32(id[j]) % kHash;; h = (h + 1) % kHash) {
                const uint32_t old = atomicCAS(&S.hash[h], ~0u, id[j]);
                if (old == ~0u) break;
                if (old == id[j]) {
                    twice = true;
                    break;
                }
            }
        }
        __syncwarp();
        twice = __any_sync(kFull, twice);
        if (twice) {
            float q[kEach];
            bool later[kEach];
#pragma unroll
            for (int j = 0; j < kEach; j++) {
                const uint32_t i = j * 32 + lane;
                q[j] = 0, later[j] = false;
                if (id[j] == ~0u) continue;
                for (uint32_t o = 0; o < P.n_listed; o++)
                    if (S.id[o] == id[j]) q[j] += S.q[o], later[j] |= o < i;
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kEach; j++) {
                S.q[j * 32 + lane] = q[j];
                if (later[j]) S.id[j * 32 + lane] = ~0u;
            }
            __syncwarp();
        }
        q_sum = warp_sum(q_sum);
        float top = -INFINITY, s = 0;
        if (P.rest) {          // the listed tokens' softmax, each once
#pragma unroll
            for (int j = 0; j < kEach; j++) top = fmaxf(top, v[j]);   // the other one where one is NaN
            top = warp_max(top);
#pragma unroll
            for (int j = 0; j < kEach; j++)
                if (top > -INFINITY && S.id[j * 32 + lane] != ~0u) s += expf(z_any(v[j], top, c));
            s = warp_sum(s);
        }
        if (lane == 0) S.q_sum = q_sum, S.twice = twice, S.m = top, S.s = s;
    }
    // The sum of q (log q - log p); with `whole`, of q (log q - log p) - q + p.
    __device__ __forceinline__ float loss(float m, float c, float log_s, bool whole) const {
        float sum = 0;
#pragma unroll
        for (int j = 0; j < kEach; j++) {
            const float q = expf(t[j]), lp = z_any(v[j], m, c) - log_s;
            if (whole) sum += id[j] == ~0u ? 0.0f : q > 0.0f ? divergence(q, t[j], lp) : expf(lp);
            else if (q > 0.0f) sum += q * (t[j] - lp);
        }
        return warp_sum(sum);
    }
};

constexpr int kSize = 4;       // vectors of a thread at a time

// The bits of vector i of the share.
template <typename T> __device__ __forceinline__ uint32_t vector_bits(const uint32_t *bits, uint32_t i) {
    const uint8_t *const bytes = (const uint8_t *)bits;
    return sizeof(T) == 2 ? bytes[i] : bytes[i / 2] >> i % 2 * 4 & 15;
}

// A vector with -infinity in the elements that `some` has bits for.
template <typename T> __device__ __forceinline__ uint4 without(uint4 q, uint32_t some) {
    constexpr uint32_t k = Bits<T>::kNegInf;
    // 16 bits: this has bit 0 at 7 and bit 1 at 15, of which prmt makes bytes (8 and 9: the sign of byte 0 or 1), and shifted
    // right by 2 the next two
    const uint32_t spread = some << 7 | some << 14;
    auto word = [=](uint32_t w, int i) {
        uint32_t mask = (uint32_t)((int32_t)(some << (31 - i)) >> 31);
        if (sizeof(T) == 2) asm("prmt.b32 %0, %1, 0, 0x9988;" : "=r"(mask) : "r"(spread >> 2 * i));
        return (w & ~mask) | (k & mask);
    };
    return make_uint4(word(q.x, 0), word(q.y, 1), word(q.z, 2), word(q.w, 3));
}

template <typename T, int kLanes, bool kTeam, bool kRest, bool kGrad>
__global__ void __launch_bounds__(kThreads<kLanes>, kCtas<kLanes>) k_distill(DistillParams P, uint32_t n_team, uint32_t n_rows, uint32_t row_bytes, uint32_t slots, bool kept) {
    constexpr int kVec = RowView<T>::kVec;
    using Tiles = Tile<T, kSize, kLanes>;
    extern __shared__ __align__(16) unsigned char smem[];
    const uint32_t r = kLanes == 32 ? blockIdx.x * kWarpRows + threadIdx.x / 32 : kTeam ? blockIdx.x / n_team : blockIdx.x;
    if (kLanes == 32 && r >= n_rows) return;
    unsigned char *const tiles = smem + (kLanes == 32 ? threadIdx.x / 32 * row_bytes : 0);
    DistillShared &S = *(DistillShared *)(tiles + slots * (Tiles::kVecs * 16));
    Team<kLanes, kTeam> team(S.team, n_team);
    team.arrive();
    const bool lists = kLanes == 32 || team.warp == kLanes / 32, reads = kLanes == 32 || !lists;
    const RowView<T> row(P.row.logits, P.row.stride, r, P.row.n_tok);
    const uint32_t vecs = row.vecs(), share = (vecs + team.size - 1) / team.size;
    const uint32_t lo = min(vecs, team.rank * share), hi = min(vecs, lo + share);
    const Feed<T, kSize, kLanes> feed(row, tiles, lo, reads ? hi : lo, kept, reads);   // under way while the entries are read
    const float c = P.row.inverse(r), c2 = usual_c<T>(c) * kLog2e;
    const float grad = kGrad ? P.d_grad ? P.d_grad[r] : P.grad : 0.0f;

    Entries list;
    if (lists) list.load<T>(P, r, row, team.lane);
    if (kRest) {
        for (uint32_t i = team.thread; i < ((hi - lo) * kVec + 31) / 32; i += kLanes == 32 ? 32 : kThreads<kLanes>) S.bits[i] = 0;
        team.sync_cta();
        if (lists)
#pragma unroll
            for (int j = 0; j < Entries::kEach; j++) {
                const uint32_t at = list.id[j] + row.shift - lo * kVec;
                if (list.id[j] != ~0u && at < (hi - lo) * kVec) atomicOr(&S.bits[at / 32], 1u << at % 32);
            }
        team.sync_cta();
    }
    if (lists) list.weigh(S, P, c, team.lane);
    if (kLanes == 32) __syncwarp();

    // The softmax of all tokens, or of the unlisted ones, whose share among themselves is exact then however little of the
    // row they hold.
    const uint32_t *const bits = S.bits;
    auto unlisted = [=](uint4 q, uint32_t i) {
        if (kRest) {
            const uint32_t some = vector_bits<T>(bits, i - lo);
            if (some) q = without<T>(q, some);
        }
        return q;
    };
    Running<T, false> sums(c2);
    const uint32_t steps = reads ? (hi - lo + Tiles::kVecs - 1) / Tiles::kVecs : 0;
    for (uint32_t n = 0; n < steps; n++) {
        Tiles t;
        feed.next(t, n);
        if (kRest) {           // what lies behind the share is -infinity whatever its bits
            uint32_t some[kSize], any = 0;
#pragma unroll
            for (int u = 0; u < kSize; u++) any |= some[u] = vector_bits<T>(S.bits, t.place(n * Tiles::kVecs, u));
            if (any) {
#pragma unroll
                for (int u = 0; u < kSize; u++) t.q[u] = without<T>(t.q[u], some[u]);
            }
        }
        const float m = t.raise_all();
        if (n == 0) sums.begin(m, c2);
        sums.add(t, m, c2);
    }
    // A row that was not kept is read again, from L2 as a rule; its first tiles come while the sums are joined.
    if (kGrad && !kept && reads) feed.start();
    float none_counted = 0.0f;
    Softmax free = softmax_join(team, sums, c2, none_counted);
    const bool fast = usual<T>(free.m, c);
    if (!fast) free = softmax_any<T, kLanes, kTeam>(team, lo, hi, c, [=](uint32_t i) { return unlisted(row.load(i), i); });

    // the whole row's softmax: m and s, and what exp of an unlisted token's z is to be multiplied by
    float m = free.m, s = free.s, to_all = 1.0f;
    if (kRest) {
        m = fmaxf(S.m, free.m);
        if (m > -INFINITY) {
            to_all = free.m > -INFINITY ? expf(z_any(free.m, m, c)) : 0.0f;
            s = free.s * to_all + (S.m > -INFINITY ? S.s * expf(z_any(S.m, m, c)) : 0.0f);
        }
    }
    const bool none = m == -INFINITY;
    const float log_s = logf(s);
    const float q_rest = kRest && free.m > -INFINITY ? fmaxf(0.0f, 1.0f - S.q_sum) : 0.0f, q_total = S.q_sum + q_rest;
    if (lists && team.rank == 0) {
        const bool whole = q_rest > 0.0f && !S.twice;   // an id listed twice has its p in two terms
        float loss = list.loss(m, c, log_s, whole);
        if (q_rest > 0.0f) {
            const float log_q = logf(q_rest), log_p = z_any(free.m, m, c) + logf(free.s) - log_s;
            loss += whole ? divergence(q_rest, log_q, log_p) : q_rest * (log_q - log_p);
        }
        if (team.lane == 0) P.loss[r] = none ? (q_total > 0.0f ? INFINITY : 0.0f) : loss;
    }
    if (!kGrad) return;

    const RowView<T> out(P.out, P.out_stride, r, P.row.n_tok);
    const bool zero = none || c == INFINITY;
    // c and grad together may be beyond 32 bits: what they are multiplied by is 0 where no token has a share, and the product too
    const float g = zero ? 0.0f : c * grad;
    const float of_free = zero || free.m == -INFINITY ? 0.0f : product(q_total / s * to_all - (q_rest > 0.0f ? q_rest / free.s : 0.0f), g);
    bool finite = fast;
    if (!(fabsf(of_free) <= 0x1p126f)) finite = false;   // as one expression 173.5 us where this takes 170.8 (8,192 x 32,256 bf16)
    const float off = __fmul_rn(free.m, c2), w = of_free * exp2_of(-fmaf(free.m, c2, -off));   // what off was rounded by
    for (uint32_t n = 0; n < steps; n++) {
        const uint32_t i0 = lo + n * Tiles::kVecs;
        Tiles t;
        if (kept) feed.again(t, n);
        else feed.next(t, n);
        const bool direct = out.shift == row.shift && Tiles::inside(row, i0, hi);
#pragma unroll
        for (int u = 0; u < kSize; u++) {
            const uint32_t i = t.place(i0, u);
            if (!direct && i >= hi) break;
            float v[kVec];
            if (finite) {
                raise<T>(t.q[u]);
                unpack(t.q[u], v, T());
#pragma unroll
                for (int e = 0; e < kVec; e += 2) {
                    const float2 x = fma2(Pair(v[e], v[e + 1]), Pair(c2, c2), Pair(-off, -off)).both();
                    const float2 d = mul2(Pair(exp2_of(x.x), exp2_of(x.y)), Pair(w, w)).both();
                    v[e] = d.x, v[e + 1] = d.y;
                }
            } else {
                unpack(t.q[u], v, T());
#pragma unroll
                for (int e = 0; e < kVec; e++) v[e] = of_free == 0.0f ? 0.0f : product(expf(z_any(v[e], free.m, c)), of_free);
            }
            put_vector(out, row, i, v, direct);
        }
    }
    team.sync_cta();
    for (uint32_t i = reads ? team.thread : P.n_listed; i < P.n_listed; i += kLanes) {
        const uint32_t id = S.id[i], at = id + row.shift - lo * kVec;
        if (id != ~0u && at < (hi - lo) * kVec)
            out.at[out.shift + id] = from_f32<T>(zero ? 0.0f : product(q_total * expf(z_any(S.v[i], m, c) - log_s) - S.q[i], g));
    }
}

// What a launch is told of its shared memory.
struct Place { uint32_t row_bytes, slots; bool kept; };

template <typename T, int kLanes, bool kTeam, bool kRest, bool kGrad>
int launch_team(bpe_ctx *ctx, const DistillParams &P, uint32_t n_rows, uint32_t team, Place at) {
    auto k = k_distill<T, kLanes, kTeam, kRest, kGrad>;
    constexpr uint32_t kRows = kLanes == 32 ? kWarpRows : 1;
    static std::atomic<uint64_t> devices{0};
    BPE_CUDA(ctx, allow_shared(k, ctx->device, kMostShared, devices), "head_distill");
    return launch_rows(ctx, "head_distill launch", k, P, (n_rows + kRows - 1) / kRows, team, kThreads<kLanes>, kTeam,
                       (size_t)at.row_bytes * kRows, n_rows, at.row_bytes, at.slots, at.kept);
}

template <typename T, bool kRest, bool kGrad> int launch(bpe_ctx *ctx, const DistillParams &P, uint32_t n_rows) {
    constexpr uint32_t kVec = RowView<T>::kVec, kAhead = Feed<T, kSize, 32>::kAhead;
    const uint32_t vecs = (P.row.n_tok + kVec - 1) / kVec + (row_shifts<T>(P.row.logits, P.row.stride, n_rows) ? 1 : 0);
    const uint32_t bytes = P.row.n_tok * (uint32_t)sizeof(T), sms = (uint32_t)ctx->sm_count;
    // A gradient's row stays in shared memory if it may, and is read once: with 266 bytes for a thread, an SM has room for
    // 24 warps.
    int least = 32;
    while (kGrad && least < kMost && bytes > 266u * least) least *= 2;
    int lanes = row_lanes(n_rows, bytes, sms, least, 40);
    if (!kGrad && lanes > 32) lanes = kMost;
    uint32_t team = 1, tile = 0;
    auto tiles = [&] { return ((vecs + team - 1) / team + tile - 1) / tile; };
    auto place = [&](bool kept) {   // of the entries, the tiles, and bits for tiles that are whole
        Place at{(uint32_t)sizeof(DistillShared), kept ? tiles() : kAhead, kept};
        at.row_bytes += at.slots * tile * 16 + (kRest ? tiles() * tile * kVec / 8 : 0);
        at.row_bytes = (at.row_bytes + 15) / 16 * 16;
        return at;
    };
    tile = kSize * lanes;
    if (lanes == 32 && place(false).row_bytes * kWarpRows > kMostShared / 2) lanes = kMost, tile = kSize * lanes;   // the bits
    const uint32_t rows = lanes == 32 ? kWarpRows : 1;
    bool kept = kGrad;
    if (lanes == kMost) {
        team = row_team(n_rows, bytes, sms, kGrad ? 4 : 2);
        if (kGrad && tiles() > kKeep) {
            // Longer rows stay where all CTAs run at once.  Else they are read again while L2 holds them: 64 MB of it for the
            // rows at hand.  (In us, read again from L2 / kept in 64 KB of more CTAs / of one CTA: 1,000 x 65,536 bf16 55 / 56 /
            // 74, with the rest 57 / 61 / 82; 1,000 x 250,000 in 4 CTAs 206 / in 8 226 with the rest, in 1 252 from DRAM.)
            const uint32_t fit = kSmShared / (place(true).row_bytes + 1024);
            kept = (uint64_t)n_rows * team <= (uint64_t)sms * (fit < 3 ? fit : 3);
            auto in_flight = [&] { const uint32_t n = 3 * sms / team; return (uint64_t)(n_rows < n ? n_rows : n) * bytes; };
            while (!kept && team < kMaxTeam && in_flight() > 64u << 20) team *= 2;
        }
    }
    kept = kept && place(true).row_bytes * rows <= kMostShared;
    while (lanes == kMost && team < kMaxTeam && place(kept).row_bytes > kMostShared) team *= 2;
    const Place at = place(kept);
    if constexpr (kGrad) {
        if (lanes == 64) return launch_team<T, 64, false, kRest, kGrad>(ctx, P, n_rows, 1, at);
        if (lanes == 128) return launch_team<T, 128, false, kRest, kGrad>(ctx, P, n_rows, 1, at);
    }
    if (lanes == 32) return launch_team<T, 32, false, kRest, kGrad>(ctx, P, n_rows, 1, at);
    return team > 1 ? launch_team<T, kMost, true, kRest, kGrad>(ctx, P, n_rows, team, at)
                    : launch_team<T, kMost, false, kRest, kGrad>(ctx, P, n_rows, 1, at);
}

template <typename T> int launch(bpe_ctx *ctx, const DistillParams &P, uint32_t n_rows) {
    if (P.rest) return P.out ? launch<T, true, true>(ctx, P, n_rows) : launch<T, true, false>(ctx, P, n_rows);
    return P.out ? launch<T, false, true>(ctx, P, n_rows) : launch<T, false, false>(ctx, P, n_rows);
}

}  // namespace
}  // namespace bpe
