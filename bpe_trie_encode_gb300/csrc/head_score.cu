// head_score.cu -- log-probabilities of given ids, with the entropy and the top
// alternatives of each row of logits, and the gradient of both.
//
// With z = (v - m) c: log s - sum(exp(z) z) / s is the entropy, so that one pass
// with two sums gives all but the alternatives; those come from the largest logit
// of each thread's tiles, noted on the way, and a second look at the few tiles that
// reach a bound.  Bound by HBM where there are many rows (8,192 x 32,256 bf16: 81 us,
// 97% of the copy rate; with 20 alternatives 98), by the latency of the steps after
// a row's last logit where there are few (256 x 65,536 bf16: 7.0 us without
// alternatives, 11.6 with 20; 1 x 32,256 bf16: 4.0 and 6.4; by graphs of calls on end).
//
// The gradient needs no sums: with the norm of the forward pass every logit's is an
// exponential and a product (with the entropy's, a fused step more).  8,192 x 32,156
// bf16: 157 us, 6.7 TB/s of reading and writing, 99% of the copy rate; 8,192 x 32,256
// 154 us, with the entropy's too.
#include "head_row.cuh"

namespace bpe {
namespace {

constexpr int kSize = 4;                   // vectors of a thread at a time
constexpr uint32_t kGradTiles = 8;         // of a CTA of the gradient, at most

struct ScoreParams {
    RowParams row;
    const int32_t *ids;
    uint32_t n_top;
    float *logprob, *entropy;
    int32_t *top_ids;
    float *top_logprob;
    float *norm;
};

// Of a row's threads, which take up to as many alternatives.
template <int kLanes> struct ScoreShared {
    static constexpr int kTop = kLanes < (int)BPE_HEAD_MAX_TOP ? kLanes : (int)BPE_HEAD_MAX_TOP;
    static constexpr int kGroups = kLanes < 256 ? 16 : 32;          // of a thread's tiles
    static constexpr int kFound = 4 * kLanes;                       // threads' groups that may hold alternatives
    static constexpr int kList = kLanes < 128 ? 8 * kLanes : 1024;  // tokens that may be among them, in the tiles' place
    static constexpr uint32_t kFeedBytes = Feed<float, kSize, kLanes>::kAhead * kSize * kLanes * 16;
    static_assert(kTop <= kLanes && (kLanes != kMost || kMaxTeam * kTop <= kList) && 2 * kList * sizeof(u64) <= kFeedBytes,
                  "one thread for each alternative, room for a team's");
    TeamShared team;
    uint32_t list_n, less_n, found_n, scan[kMostWarps];
    float bound[kMostWarps];
    u64 best[kTop];                        // in order
    uint32_t found[kFound];
    uint16_t most[kGroups][kLanes];        // the largest logit of each
};
// Shared memory of a row: its tiles, and without alternatives the team's part alone.
template <int kLanes, bool kTops>
constexpr uint32_t kScoreBytes = ScoreShared<kLanes>::kFeedBytes + (uint32_t)(kTops ? sizeof(ScoreShared<kLanes>) : sizeof(TeamShared));

__device__ __forceinline__ u64 entry_of(uint32_t key, uint32_t id) { return (u64)key << 32 | (uint32_t)~id; }

// The alternatives in `list`, at most k of this CTA's, for any logits: the key of the k-th largest is found by bits, two
// a pass (of bf16 8 passes, f16 10, f32 16, and three more reads of the row: 256 x 32,256, all equal, 20 alternatives, 93 / 109 /
// 168 us); those above it are listed, and as many of its equals, in order of ids, as there is room for.  `have` >= 0: the lists
// hold all logits above kLow, so many, and fewer than k; then there may be no more, or those that a mask has set to one value,
// the largest of the others (256 x 32,256 bf16 with 5 others, 20 alternatives: 93 us by bits, 20 so; masks above kLow, -1e4 and
// -1e9, go by bits).  Gives the team's turn.
template <typename T, int kLanes, bool kTeam>
__device__ __noinline__ int list_any(ScoreShared<kLanes> &S, u64 *list, Team<kLanes, kTeam> team, RowView<T> row, uint32_t lo, uint32_t hi,
                                     uint32_t k, float have) {
    constexpr int kVec = RowView<T>::kVec, kShift = Bits<T>::kShift, kBits = (32 - kShift + 1) & ~1;
    uint32_t some = 0;
    float low = -INFINITY;                 // the largest at or below kLow
    for (uint32_t i = lo + team.thread; i < hi; i += kLanes) {
        float v[kVec];
        unpack(row.load(i), v, T());
#pragma unroll
        for (int e = 0; e < kVec; e++) some += v[e] > -INFINITY, low = v[e] <= Usual<T>::kLow ? fmaxf(low, v[e]) : low;
    }
    const float valid = team.sum(make_float4(some, 0, 0, 0)).x;   // counts up to 2^22 are exact in 32 bits
    const float want = fminf((float)k, valid);
    if (want == have) return team.turn;
    uint32_t cut = 0;
    float4 n;
    float above_all = -1.0f;
    if (have >= 0.0f && (low = team.max(low)) > -INFINITY) {
        cut = key_of(low) >> kShift;
        uint32_t equal = 0;
        for (uint32_t i = lo + team.thread; i < hi; i += kLanes) {
            float v[kVec];
            unpack(row.load(i), v, T());
#pragma unroll
            for (int e = 0; e < kVec; e++) equal += key_of(v[e]) >> kShift == cut;
        }
        n = team.sum(make_float4(0, equal, 0, 0));
        if (have + n.y >= want) above_all = have;
    }
    if (above_all < 0.0f) {
        if (team.thread == 0) S.list_n = 0;
        team.sync_cta();
        if (want == 0.0f) return team.turn;
        cut = 0;
        for (int bit = kBits - 2; bit >= 0; bit -= 2) {
            uint32_t n1 = 0, n2 = 0, n3 = 0;
            for (uint32_t i = lo + team.thread; i < hi; i += kLanes) {
                float v[kVec];
                unpack(row.load(i), v, T());
#pragma unroll
                for (int e = 0; e < kVec; e++) {
                    const uint32_t key = key_of(v[e]) >> kShift;
                    n1 += key >= (cut | 1u << bit), n2 += key >= (cut | 2u << bit), n3 += key >= (cut | 3u << bit);
                }
            }
            const float4 c = team.sum(make_float4(n1, n2, n3, 0));
            cut |= (c.z >= want ? 3u : c.y >= want ? 2u : c.x >= want ? 1u : 0u) << bit;
        }
        uint32_t above = 0, equal = 0;
        for (uint32_t i = lo + team.thread; i < hi; i += kLanes) {
            float v[kVec];
            unpack(row.load(i), v, T());
#pragma unroll
            for (int e = 0; e < kVec; e++) {
                const uint32_t key = key_of(v[e]);
                if (key >> kShift > cut) list[atomicAdd(&S.list_n, 1)] = entry_of(key, i * kVec + e - row.shift), above++;   // fewer than k
                equal += key >> kShift == cut;
            }
        }
        n = team.sum(make_float4(above, equal, 0, 0));
        above_all = n.x;
    }
    uint32_t mine = 0, before = 0;         // equals of this CTA, and of those before it
    if (kTeam) {
        for (uint32_t r = 0; r < team.rank; r++) before += (uint32_t)team.S.slot[team.turn][r].y;
        mine = (uint32_t)team.S.slot[team.turn][team.rank].y;
    } else {
        mine = (uint32_t)n.y;
    }
    const uint32_t need = (uint32_t)(want - above_all);
    const uint32_t quota = min(mine, need > before ? need - before : 0u);
    uint32_t seen = 0;
    for (uint32_t i0 = lo; i0 < hi && seen < quota; i0 += kLanes) {
        const uint32_t i = i0 + team.thread;
        float v[kVec];
        uint32_t own = 0;
        if (i < hi) {
            unpack(row.load(i), v, T());
#pragma unroll
            for (int e = 0; e < kVec; e++) own += key_of(v[e]) >> kShift == cut;
        }
        const uint32_t upto = warp_incl_sum(own, team.lane);
        uint32_t at = seen + upto - own;
        if (kLanes == 32) {
            seen += __shfl_sync(kFull, upto, 31);
        } else {
            __syncthreads();
            if (team.lane == 31) S.scan[team.warp] = upto;
            __syncthreads();
            for (int w = 0; w < kLanes / 32; w++) {
                if (w < team.warp) at += S.scan[w];
                seen += S.scan[w];
            }
        }
        if (own) {
#pragma unroll
            for (int e = 0; e < kVec; e++)
                if (key_of(v[e]) >> kShift == cut && at++ < quota)
                    list[atomicAdd(&S.list_n, 1)] = entry_of(key_of(v[e]), i * kVec + e - row.shift);
        }
    }
    team.sync_cta();
    return team.turn;
}

// Rows are many where they have few threads each (row_lanes): instructions count, not a row's latency.
template <int kLanes> constexpr bool kManyRows = kLanes < 256;

// 32 kEach entries in order, largest first, by a bitonic network: entry e of a lane is number 32 e + lane.
template <int kEach> __device__ __forceinline__ void sort_warp(u64 (&v)[kEach], int lane) {
#pragma unroll
    for (int size = 2; size <= 32 * kEach; size <<= 1)
#pragma unroll
        for (int d = size >> 1; d > 0; d >>= 1)
#pragma unroll
            for (int e = 0; e < kEach; e++) {
                if (d >= 32) {
                    const int o = e ^ d / 32;
                    if (o < e) continue;
                    const bool down = (32 * e & size) == 0;
                    const u64 a = v[e], b = v[o];
                    const bool swap = (a < b) == down;
                    v[e] = swap ? b : a, v[o] = swap ? a : b;
                } else {
                    const u64 o = __shfl_xor_sync(kFull, v[e], d);
                    const bool first = (lane & d) == 0, down = ((32 * e + lane) & size) == 0;
                    v[e] = (first == down) == (v[e] < o) ? o : v[e];
                }
            }
}
// f(place, entry) for the list's k largest, by one warp.
template <int kEach, typename F> __device__ __forceinline__ void sort_list(const u64 *list, uint32_t n, uint32_t k, int lane, F f) {
    u64 v[kEach];
#pragma unroll
    for (int e = 0; e < kEach; e++) v[e] = 32 * e + lane < n ? list[32 * e + lane] : 0;
    sort_warp(v, lane);
#pragma unroll
    for (int e = 0; e < kEach; e++)
        if (32 * e + lane < min(n, k)) f(32 * e + lane, v[e]);
}
// The same for any list, by all of a row's threads: a place is the number of larger entries, counted by four threads for each.
// Where rows are many, up to 128 entries are sorted by one warp: fewer instructions, but one after the other (64 alternatives,
// sorted / ranked: 8,192 x 32,256 bf16 by 128 threads 123 / 137 us; 256 x 65,536 by 256 14.7 / 13.4).
template <int kLanes, bool kTeam, typename F>
__device__ __forceinline__ uint32_t rank_list(const Team<kLanes, kTeam> &team, const u64 *list, uint32_t n, uint32_t k, F f) {
    if (kManyRows<kLanes> && n <= 128) {
        if (team.warp == 0) {
            if (n <= 32) sort_list<1>(list, n, k, team.lane, f);
            else if (n <= 64) sort_list<2>(list, n, k, team.lane, f);
            else sort_list<4>(list, n, k, team.lane, f);
        }
        return min(n, k);
    }
    const uint32_t part = team.thread & 3;
    for (uint32_t i0 = 0; i0 + (team.thread & ~31u) / 4 < n; i0 += kLanes / 4) {
        const uint32_t i = i0 + team.thread / 4;
        const u64 one = list[min(i, n - 1)];
        uint32_t place = 0;
        for (uint32_t j = part; j < n; j += 4) place += list[j] > one;
        place += __shfl_xor_sync(kFull, place, 1);
        place += __shfl_xor_sync(kFull, place, 2);
        if (i < n && part == 0 && place < k) f(place, one);
    }
    return min(n, k);
}

// ------------------------------------------- alternatives, on the way ---
// While a row goes by, every thread notes the largest logit of each of its tiles (or of up to kGroups groups of them).  Then
// comes a bound from below on the k-th largest logit of the CTA's share: with the j-th largest of each warp's 32 largest logits
// in S.bound, and w j >= k of them, the least of w warps' bounds has k logits at or above it.  The groups that reach it, some
// 1.5 k where likely tokens lie anywhere in the row, are read once more, and what reaches it of them is ranked.  Where all lie
// near each other at its start the warp that has none of them sets the bound, and more reach it (256 x 65,536 bf16, 20
// alternatives, logits of -log(1 + id) and normal noise of 1 / 0.7 / 0.3: 14.7 / 15.7 / 151 us, the last by bits, where those
// spread take 12.5).  (Listing on the way, with a bound that rises, cost 80 to 280 instructions a tile of 193: 256 x 65,536
// bf16, 20 alternatives, 13.7 us.)
template <int kLanes> struct Bound {
    uint32_t warps, j;                     // 0 warps: the share is too short for one

    __device__ __forceinline__ Bound(uint32_t vecs, uint32_t k) : warps(min((uint32_t)kLanes / 32, vecs / 32)), j(0) {
        if (warps) j = (k + warps - 1) / warps;
        if (j > 32) warps = 0;
    }
    __device__ __forceinline__ float least(const ScoreShared<kLanes> &S, float low) const {
        if (!warps) return low;
        float b = INFINITY;
        for (uint32_t w = 0; w < warps; w++) b = fminf(b, S.bound[w]);
        return b;
    }
    // this warp's, from its lanes' largest logits: by taking out the largest where few are asked for, by sorting else
    __device__ __forceinline__ void write(ScoreShared<kLanes> &S, float v, int lane, int warp) const {
        if (warp >= (int)warps) return;
        if (j <= 8) {
            uint32_t key = key_of(v), top = 0;
            for (uint32_t i = 0; i < j; i++) {
                top = __reduce_max_sync(kFull, key);
                if (lane == __ffs(__ballot_sync(kFull, key == top)) - 1) key = 0;
            }
            if (lane == 0) S.bound[warp] = key_value(top);
            return;
        }
#pragma unroll
        for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
            for (int d = size >> 1; d > 0; d >>= 1) {
                const float o = __shfl_xor_sync(kFull, v, d);
                const bool first = (lane & d) == 0, down = (lane & size) == 0 || size == 32;   // largest first
                v = first == down ? fmaxf(v, o) : fminf(v, o);
            }
        if (lane == (int)j - 1) S.bound[warp] = v;
    }
};

// A group's largest logit in 16 bits, no less than it is.
__device__ __forceinline__ uint16_t note(float v, float) { return __bfloat16_as_ushort(__float2bfloat16_ru(v)); }
__device__ __forceinline__ uint16_t note(float v, __nv_bfloat16) { return (uint16_t)(__float_as_uint(v) >> 16); }
__device__ __forceinline__ uint16_t note(float v, __half) { return __half_as_ushort(__float2half_rn(v)); }
__device__ __forceinline__ float noted(uint16_t b, float) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float noted(uint16_t b, __nv_bfloat16) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ float noted(uint16_t b, __half) { return __half2float(__ushort_as_half(b)); }

// This thread's groups that reach the bound.
template <typename T, int kLanes>
__device__ __forceinline__ void find(ScoreShared<kLanes> &S, uint32_t groups, float bound) {
    const uint32_t t = row_thread<kLanes>();
    for (uint32_t g = 0; g < groups; g++) {
        const float m = noted(S.most[g][t], T());
        if (m >= bound && m > Usual<T>::kLow) {
            const uint32_t at = atomicAdd(&S.found_n, 1);
            if (at < S.kFound) S.found[at] = g << 16 | t;
        }
    }
}

// The logits of a vector that reach it, to the list.
template <typename T, int kLanes>
__device__ __forceinline__ void list_vector(ScoreShared<kLanes> &S, u64 *list, const RowView<T> &row, uint4 q, uint32_t place, float bound) {
    constexpr int kVec = RowView<T>::kVec;
    float v[kVec];
    unpack(q, v, T());
    uint32_t some = 0;
#pragma unroll
    for (int e = 0; e < kVec; e++) some |= v[e] >= bound && v[e] > Usual<T>::kLow ? 1u << e : 0u;
    if (!some) return;
    uint32_t at = atomicAdd(&S.list_n, __popc(some));
#pragma unroll
    for (int e = 0; e < kVec; e++)
        if (some >> e & 1) {
            if (at < S.kList) list[at] = entry_of(key_of(v[e]), place * kVec - row.shift + e);
            at++;
        }
}
// Those of the groups that were found.  A thread takes a vector, or where rows are many a group, tile by tile, of which it looks
// closer at the vectors that have any (one, as a rule).
template <typename T, int kLanes>
__device__ __forceinline__ void list_found(ScoreShared<kLanes> &S, u64 *list, const RowView<T> &row, uint32_t lo, uint32_t hi, uint32_t tiles,
                                           float bound) {
    const uint32_t n = min(S.found_n, (uint32_t)S.kFound), each = tiles * kSize;
    if (!kManyRows<kLanes>) {
        for (uint32_t i = row_thread<kLanes>(); i < n * each; i += kLanes) {
            const uint32_t f = S.found[i / each], place = lo + ((f >> 16) * each + i % each) * kLanes + (f & 0xFFFFu);
            if (place < hi) list_vector<T, kLanes>(S, list, row, row.load(place), place, bound);
        }
        return;
    }
    for (uint32_t i = row_thread<kLanes>(); i < n; i += kLanes) {
        const uint32_t f = S.found[i];
        for (uint32_t t = 0; t < tiles; t++) {
            const uint32_t first = lo + ((f >> 16) * each + t * kSize) * kLanes + (f & 0xFFFFu);
            uint4 q[kSize];
#pragma unroll
            for (int u = 0; u < kSize; u++) q[u] = first + u * kLanes < hi ? row.load(first + u * kLanes) : Tile<T, kSize, kLanes>::fill();
            uint32_t some = 0;
#pragma unroll
            for (int u = 0; u < kSize; u++) {
                const float m = Words<T>::largest(raise<T>(q[u]));
                some |= m >= bound && m > Usual<T>::kLow ? 1u << u : 0u;
            }
            while (some) {
                const int u = __ffs(some) - 1;
                some &= some - 1;
                uint4 one = q[0];
#pragma unroll
                for (int o = 1; o < kSize; o++)
                    if (u == o) one = q[o];
                list_vector<T, kLanes>(S, list, row, one, first + u * kLanes, bound);
            }
        }
    }
}

// A list that is long (a short row's, of which no tiles were left out) without what is below a bound of its own, in the place
// behind it (283 x 402 f16, 57 alternatives: 20 us with all pairs of 402 ranked, 8.6 so).
template <int kLanes, bool kTeam>
__device__ __forceinline__ uint32_t shorten(ScoreShared<kLanes> &S, const Team<kLanes, kTeam> &team, u64 *list, uint32_t n, uint32_t k) {
    u64 most = 0;
    for (uint32_t i = team.thread; i < n; i += kLanes) most = max(most, list[i]);
    const Bound<kLanes> tops(n, k);
    if (team.thread == 0) S.less_n = 0;
    tops.write(S, most ? key_value((uint32_t)(most >> 32)) : -INFINITY, team.lane, team.warp);
    team.sync_cta();
    const u64 least = (u64)key_of(tops.least(S, -INFINITY)) << 32;
    for (uint32_t i = team.thread; i < n; i += kLanes)
        if (list[i] >= least) list[S.kList + atomicAdd(&S.less_n, 1)] = list[i];
    team.sync_cta();
    return S.less_n;
}

template <typename T, int kLanes, bool kTeam, bool kTops>
__global__ void __launch_bounds__(kLanes == 32 ? kWarpRows * 32 : kLanes, kLanes == 32 ? 4 : 1024 / kLanes) k_logprobs(ScoreParams P, uint32_t n_team, uint32_t n_rows) {
    using Tiles = Tile<T, kSize, kLanes>;
    using Shared = ScoreShared<kLanes>;
    extern __shared__ __align__(16) unsigned char smem[];
    const uint32_t r = kLanes == 32 ? blockIdx.x * kWarpRows + threadIdx.x / 32 : kTeam ? blockIdx.x / n_team : blockIdx.x;
    if (kLanes == 32 && r >= n_rows) return;
    unsigned char *const tiles = smem + (kLanes == 32 ? threadIdx.x / 32 * kScoreBytes<kLanes, kTops> : 0);
    Shared &S = *(Shared *)(tiles + Shared::kFeedBytes);
    Team<kLanes, kTeam> team(S.team, n_team);
    team.arrive();
    const RowView<T> row(P.row.logits, P.row.stride, r, P.row.n_tok);
    const uint32_t vecs = row.vecs(), share = (vecs + team.size - 1) / team.size;
    const uint32_t lo = min(vecs, team.rank * share), hi = min(vecs, lo + share);
    const float c = P.row.inverse(r), c2 = usual_c<T>(c) * kLog2e;
    const uint32_t k = kTops ? P.n_top : 0;
    int32_t id = -1;
    float given = 0.0f;
    if (team.thread == 0 && team.rank == 0 && P.logprob) {
        id = P.ids[r];
        if (id >= 0 && (uint32_t)id < P.row.n_tok) given = to_f32(row.at[row.shift + id]);
    }

    const Feed<T, kSize, kLanes> feed(row, tiles, lo, hi);
    Running<T, true> sums(c2);
    const Bound<kLanes> tops(hi - lo, k);
    float count = 0.0f;
    u64 *const list = (u64 *)tiles;        // once the tiles are through
    if (kTops) {
        if (team.thread == 0) S.list_n = S.found_n = 0;
        const uint32_t steps = feed.steps(), per = (steps + S.kGroups - 1) / S.kGroups;   // tiles of a group
        uint32_t group = 0, left = per;
        float most = Usual<T>::kLow;
        for (uint32_t n = 0; n < steps; n++) {
            Tiles t;
            feed.next(t, n);
            const float m = t.raise_all();
            if (n == 0) sums.begin(m, c2);
            sums.add(t, m, c2);
            most = fmaxf(most, m);
            if (--left == 0 || n + 1 == steps) {
                S.most[group++][team.thread] = note(most, T());
                left = per, most = Usual<T>::kLow;
            }
        }
        tops.write(S, sums.most, team.lane, team.warp);
        team.sync_cta();
        const float bound = tops.least(S, Usual<T>::kLow);
        find<T, kLanes>(S, group, bound);
        team.sync_cta();
        list_found<T, kLanes>(S, list, row, lo, hi, per, bound);
        team.sync_cta();
        const bool over = S.found_n > S.kFound || S.list_n > S.kList;
        count = over ? -0x1p24f : fminf((float)S.list_n, (float)k);
    } else {
        for (uint32_t n = 0, i0 = lo; i0 < hi; i0 += Tiles::kVecs, n++) {
            Tiles t;
            feed.next(t, n);
            const float m = t.raise_all();
            if (n == 0) sums.begin(m, c2);
            sums.add(t, m, c2);
        }
    }
    Softmax all = softmax_join(team, sums, c2, count);
    if (kLanes > 32 && !kTeam && !kTops && team.warp > 0 && usual<T>(all.m, c)) return;
    if (!usual<T>(all.m, c)) all = softmax_any<T, kLanes, kTeam>(team, lo, hi, c, [=](uint32_t i) { return row.load(i); });
    // more equal or masked logits than the list holds, or fewer others than were asked for
    if (kTops && count < (float)min(k, P.row.n_tok)) team.turn = list_any<T, kLanes, kTeam>(S, list, team, row, lo, hi, k, count);

    const bool none = all.m == -INFINITY;
    const float log_s = none ? 0.0f : logf(all.s);
    if (team.thread == 0 && team.rank == 0) {
        if (P.norm) P.norm[2 * (uint64_t)r] = all.m, P.norm[2 * (uint64_t)r + 1] = log_s;
        if (P.entropy) P.entropy[r] = none ? 0.0f : log_s - all.sz / all.s;
        if (P.logprob) P.logprob[r] = id < 0 || (uint32_t)id >= P.row.n_tok ? 0.0f : none ? -INFINITY : z_any(given, all.m, c) - log_s;
    }
    if (!kTops) return;
    auto put = [=](uint32_t place, u64 one) {
        const uint64_t at = (uint64_t)r * k + place;
        if (P.top_ids) P.top_ids[at] = (int32_t)~(uint32_t)one;
        if (P.top_logprob) P.top_logprob[at] = z_any(key_value((uint32_t)(one >> 32)), all.m, c) - log_s;
    };
    uint32_t total, listed = S.list_n;
    const u64 *from = list;
    if (listed > 128) listed = shorten(S, team, list, listed, k), from += S.kList;
    if (!kTeam) {
        total = rank_list(team, from, listed, k, put);
    } else {
        const uint32_t n = rank_list(team, from, listed, k, [&](uint32_t place, u64 one) { S.best[place] = one; });
        __syncthreads();
        const u64 one = S.best[min(team.thread, k - 1)];   // this thread's, of the n
        team.exchange(make_float4((float)n, 0, 0, 0));
        total = 0;
        for (uint32_t o = 0; o < team.size; o++) total += (uint32_t)team.S.slot[team.turn][o].x;
        // every CTA's list, then each of its own finds its place by those that are larger
        for (uint32_t o = 0; o < team.size; o++)
            if (o != team.rank && team.thread < (uint32_t)team.S.slot[team.turn][o].x) list[o * k + team.thread] = far_load(&S.best[team.thread], o);
        __syncthreads();
        uint32_t place = team.thread;
        if (team.thread < n)
            for (uint32_t o = 0; o < team.size; o++) {
                if (o == team.rank) continue;
                uint32_t x = 0, y = (uint32_t)team.S.slot[team.turn][o].x;
                while (x < y) {
                    const uint32_t mid = (x + y) / 2;
                    if (list[o * k + mid] > one) x = mid + 1;
                    else y = mid;
                }
                place += x;
            }
        if (team.thread < n && place < k) put(place, one);
    }
    if (team.rank == 0 && team.thread >= total && team.thread < k) {
        const uint64_t at = (uint64_t)r * k + team.thread;
        if (P.top_ids) P.top_ids[at] = -1;
        if (P.top_logprob) P.top_logprob[at] = -INFINITY;
    }
    team.arrive();
    team.wait();   // the others have read this CTA's list
}

// ----------------------------------------------------------- gradient ---
struct ScoreGradParams {
    RowParams row;
    const int32_t *ids;
    const float *norm, *grad_logprob, *entropy, *grad_entropy;
    void *out;
    uint64_t out_stride;
};

// No sums, so that a row is cut where it suits: a CTA takes `each` tiles of it.
template <typename T, int kLanes, bool kEntropy>
__global__ void __launch_bounds__(256) k_logprobs_backward(ScoreGradParams P, uint32_t cuts, uint32_t each, uint32_t n_rows) {
    constexpr int kVec = RowView<T>::kVec;
    using Tiles = Tile<T, kSize, kLanes>;
    extern __shared__ __align__(16) unsigned char tiles[];
    const uint32_t unit = kLanes == 32 ? blockIdx.x * kWarpRows + threadIdx.x / 32 : blockIdx.x, r = unit / cuts, cut = unit % cuts;
    if (r >= n_rows) return;
    const RowView<T> row(P.row.logits, P.row.stride, r, P.row.n_tok), out(P.out, P.out_stride, r, P.row.n_tok);
    const uint32_t lo = cut * each * Tiles::kVecs, hi = min(row.vecs(), lo + each * Tiles::kVecs);
    if (lo >= hi) return;
    using F = Feed<T, kSize, kLanes>;
    const F feed(row, tiles + (kLanes == 32 ? threadIdx.x / 32 * (F::kAhead * F::kBytes) : 0), lo, hi);
    const float c = P.row.inverse(r);
    const float m = P.norm[2 * (uint64_t)r], log_s = P.norm[2 * (uint64_t)r + 1];
    const int32_t id = P.ids ? P.ids[r] : -1;
    const bool given = id >= 0 && (uint32_t)id < P.row.n_tok;
    const float a = given && P.grad_logprob ? P.grad_logprob[r] : 0.0f;
    const float b = kEntropy ? P.grad_entropy[r] : 0.0f, h = kEntropy ? P.entropy[r] : 0.0f;
    const bool zero = m == -INFINITY || c == INFINITY;
    // x = exp2(z) of the logits relative to R, m c log2 e rounded; d = x (f + g z), and c a more for the id itself.  The
    // factor 1 / s, and what R was rounded by, are part of f and g.
    const float c2 = c * kLog2e, off = __fmul_rn(m, c2), d0 = fmaf(m, c2, -off);
    const float w = c * exp2_of(-fmaf(log_s, kLog2e, d0));
    const float f = -w * (a + b * (h - log_s - d0 * kLn2)), g = -w * b * kLn2;
    // A masked logit's x is 0, and its z kLow c2 - R: f + g z is to be finite, or 0 times it is NaN.
    const bool fast = usual<T>(m, c) && fabsf(f) + fabsf(g) * fmaf(-Usual<T>::kLow, c2, fabsf(off)) <= 0x1p126f;
    const Pair c22(c2, c2), off2(-off, -off), f2(f, f), g2(g, g);
    const uint32_t hot = given ? row.shift + (uint32_t)id : ~0u;
    for (uint32_t n = 0; n * Tiles::kVecs < hi - lo; n++) {
        Tiles t;
        feed.next(t, n);
        const bool direct = out.shift == row.shift && Tiles::inside(row, lo + n * Tiles::kVecs, hi);
#pragma unroll
        for (int u = 0; u < kSize; u++) {
            const uint32_t i = t.place(lo + n * Tiles::kVecs, u);
            if (!direct && i >= hi) break;
            float v[kVec];
            if (fast) {
                raise<T>(t.q[u]);
                unpack(t.q[u], v, T());
#pragma unroll
                for (int e = 0; e < kVec; e += 2) {
                    const Pair z = fma2(Pair(v[e], v[e + 1]), c22, off2);
                    const float2 x = z.both();
                    const float2 d = mul2(Pair(exp2_of(x.x), exp2_of(x.y)), kEntropy ? fma2(g2, z, f2) : f2).both();
                    v[e] = d.x, v[e + 1] = d.y;
                }
            } else {
                unpack(t.q[u], v, T());
#pragma unroll
                for (int e = 0; e < kVec; e++) {
                    const float lp = z_any(v[e], m, c) - log_s, p = expf(lp), one = i * kVec + e == hot ? a : 0.0f;
                    v[e] = zero ? 0.0f : c * (one - a * p - (p > 0.0f ? b * p * (lp + h) : 0.0f));
                }
            }
            if (fast && i == hot / kVec) {
#pragma unroll
                for (int e = 0; e < kVec; e++) v[e] = fmaf(c, e == hot % kVec ? a : 0.0f, v[e]);
            }
            put_vector(out, row, i, v, direct);
        }
    }
}

template <typename T, int kLanes, bool kTeam, bool kTops>
int launch_team(bpe_ctx *ctx, const ScoreParams &P, uint32_t n_rows, uint32_t team) {
    auto k = k_logprobs<T, kLanes, kTeam, kTops>;
    constexpr uint32_t kRows = kLanes == 32 ? kWarpRows : 1, kShared = kScoreBytes<kLanes, kTops> * kRows;
    static std::atomic<uint64_t> devices{0};
    BPE_CUDA(ctx, allow_shared(k, ctx->device, kShared, devices), "head_logprobs");
    return launch_rows(ctx, "head_logprobs launch", k, P, (n_rows + kRows - 1) / kRows, team, kLanes * kRows, kTeam, kShared, n_rows);
}
// Whether a row has a CTA of 512 threads: where no SM has more than one row, and they are long.  In us, 512 threads / clusters
// of two CTAs of 256, 20 alternatives: 120 x 65,536 bf16 9.4 / 11.0, 152 x 250,000 bf16 17.8 / 19.7; 120 x 32,256 8.4 / 7.5.
static bool row_wide(uint32_t n_rows, uint32_t bytes, uint32_t sms) { return n_rows <= sms && n_rows > sms / 2 && bytes >= 65536; }

template <typename T> int launch_logprobs(bpe_ctx *ctx, const ScoreParams &P, uint32_t n_rows) {
    const uint32_t bytes = P.row.n_tok * (uint32_t)sizeof(T), sms = (uint32_t)ctx->sm_count, team = row_team(n_rows, bytes, sms, 2);
    const bool wide = row_wide(n_rows, bytes, sms);
    if (!P.n_top || !(P.top_ids || P.top_logprob)) {
        if (row_lanes(n_rows, bytes, sms, 32, 40) == 32) return launch_team<T, 32, false, false>(ctx, P, n_rows, 1);
        if (wide) return launch_team<T, 512, false, false>(ctx, P, n_rows, 1);
        return team > 1 ? launch_team<T, kMost, true, false>(ctx, P, n_rows, team) : launch_team<T, kMost, false, false>(ctx, P, n_rows, 1);
    }
    // The threads are the groups of Bound: with fewer than 1.5 for each alternative the bound leaves more than the list holds.
    int least = 32;
    while (least < kMost && (uint32_t)least * 2 < P.n_top * 3) least *= 2;
    switch (row_lanes(n_rows, bytes, sms, least, 4)) {
    case 32: return launch_team<T, 32, false, true>(ctx, P, n_rows, 1);
    case 64: return launch_team<T, 64, false, true>(ctx, P, n_rows, 1);
    case 128: return launch_team<T, 128, false, true>(ctx, P, n_rows, 1);
    default:
        if (wide) return launch_team<T, 512, false, true>(ctx, P, n_rows, 1);
        return team > 1 ? launch_team<T, kMost, true, true>(ctx, P, n_rows, team) : launch_team<T, kMost, false, true>(ctx, P, n_rows, 1);
    }
}

// A CTA takes up to eight tiles of a row, as long as 16 CTAs an SM are left: what a row costs once is shared by its tiles, and many
// CTAs leave a short last wave.  (Us where 1 / 4 / 16 / 64 are to be left, and with one tile each: 8,192 x 32,156 bf16 155 / 155 / 155 / 154 /
// 165; 8,192 x 4,352 22.9 / 22.7 / 25.9 / 29.0 / 29.2; 500 x 65,536 20.5 / 19.9 / 22.6 / 22.5 / 22.5; 300 x 32,256 5.7 / 7.0 /
// 6.7 / 6.7 / 6.8; 1,024 x 250,000 f16 153 / 153 / 153 / 148 / 147.)
template <typename T, int kLanes> int launch_backward(bpe_ctx *ctx, const ScoreGradParams &P, uint32_t n_rows) {
    using F = Feed<T, kSize, kLanes>;
    constexpr uint32_t kRows = 256 / kLanes, kVec = RowView<T>::kVec;
    const uint32_t vecs = (P.row.n_tok + kVec - 1) / kVec + (row_shifts<T>(P.row.logits, P.row.stride, n_rows) ? 1 : 0);
    const uint32_t tiles = (vecs + F::Tiles::kVecs - 1) / F::Tiles::kVecs;
    uint32_t each = 1;
    while (each < kGradTiles && each < tiles && (uint64_t)n_rows * ((tiles + each) / (each + 1)) >= 16ull * kRows * ctx->sm_count) each++;
    const uint32_t cuts = (tiles + each - 1) / each;
    const uint64_t ctas = ((uint64_t)n_rows * cuts + kRows - 1) / kRows;
    if (ctas > 0x7FFFFFFFu) return fail(ctx, BPE_ERR_INVALID_ARG, "head_logprobs_backward: too many rows");
    auto k = P.grad_entropy ? k_logprobs_backward<T, kLanes, true> : k_logprobs_backward<T, kLanes, false>;
    k<<<(uint32_t)ctas, 256, F::kAhead * F::kBytes * kRows, ctx->stream>>>(P, cuts, each, n_rows);
    BPE_CUDA(ctx, cudaGetLastError(), "head_logprobs_backward launch");
    return BPE_OK;
}
// A warp a row where rows are many and no more than five of a warp's tiles; a CTA's tile is 16 KB, of which a short row leaves
// most threads idle, and few rows leave SMs idle if they are warps.  (Us by warps / CTAs, bf16: 64 x 1,000 2.9 / 2.4, 512 x 1,000
// 3.1 / 3.4, 4,096 x 1,000 4.7 / 12.4, 4,096 x 5,000 13.1 / 17.0, 256 x 5,000 3.1 / 3.1, 4,096 x 8,000 25.4 / 25.2.)
template <typename T> int launch_backward(bpe_ctx *ctx, const ScoreGradParams &P, uint32_t n_rows) {
    return n_rows >= 256 && P.row.n_tok * sizeof(T) <= 10240 ? launch_backward<T, 32>(ctx, P, n_rows) : launch_backward<T, kMost>(ctx, P, n_rows);
}

}  // namespace

int head_row_check(bpe_ctx *ctx, const char *name, const void *d_logits, uint64_t stride, int type, uint32_t n_rows,
                   uint32_t n_tok) {
    if (!head_type_ok(type)) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: unknown element type", name);
    if (n_tok == 0 || n_tok > BPE_HEAD_MAX_TOKENS)
        return fail(ctx, BPE_ERR_INVALID_ARG, "%s: %u tokens outside 1..%u", name, n_tok, BPE_HEAD_MAX_TOKENS);
    if (n_rows > 0x7FFFFFFFu) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: %u rows", name, n_rows);
    if (n_rows && !d_logits) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (n_rows && (uintptr_t)d_logits % head_type_size(type))
        return fail(ctx, BPE_ERR_INVALID_ARG, "%s: logits that do not start on an element", name);
    if (n_rows > 1 && stride < n_tok) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: the row stride is below n_tok", name);
    return BPE_OK;
}

int head_grad_check(bpe_ctx *ctx, const char *name, const void *d_logits, uint64_t stride, int type, uint32_t n_rows,
                    uint32_t n_tok, const void *d_grad, uint64_t grad_stride) {
    if (n_rows == 0) return BPE_OK;
    if (!d_grad) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: null pointer", name);
    const size_t e = head_type_size(type);
    if ((uintptr_t)d_grad % e) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: a gradient that does not start on an element", name);
    if (n_rows > 1 && grad_stride < n_tok)
        return fail(ctx, BPE_ERR_INVALID_ARG, "%s: the gradient's row stride is below n_tok", name);
    // The rows of the two may interleave (columns of one buffer), but no row's bytes may be another's: with equal strides the
    // distance of the two within a row's period decides; with others the whole ranges must be apart.
    const uintptr_t x = (uintptr_t)d_logits, y = (uintptr_t)d_grad;
    if (x == y && (n_rows == 1 || stride == grad_stride)) return BPE_OK;
    const uint64_t xs = n_rows > 1 ? stride : n_tok, ys = n_rows > 1 ? grad_stride : n_tok;
    const uintptr_t xe = x + ((uint64_t)(n_rows - 1) * xs + n_tok) * e, ye = y + ((uint64_t)(n_rows - 1) * ys + n_tok) * e;
    bool apart = xe <= y || ye <= x;
    if (!apart && n_rows > 1 && xs == ys) {
        const uint64_t period = xs * e, off = y >= x ? (y - x) % period : (period - (x - y) % period) % period;
        apart = off >= (uint64_t)n_tok * e && off + (uint64_t)n_tok * e <= period;
    }
    if (!apart) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: the gradient overlaps the logits, and is not the logits themselves", name);
    return BPE_OK;
}

}  // namespace bpe

using namespace bpe;

extern "C" int head_logprobs(bpe_ctx *ctx, const void *d_logits, uint64_t stride, int type, uint32_t n_rows, uint32_t n_tok,
                             const int32_t *d_ids, float temperature, const float *d_temperature, uint32_t n_top,
                             float *d_logprob_out, float *d_entropy_out, int32_t *d_top_ids_out, float *d_top_logprob_out,
                             float *d_norm_out) {
    if (!ctx) return BPE_ERR_INVALID_ARG;
    if (const int rc = head_row_check(ctx, "head_logprobs", d_logits, stride, type, n_rows, n_tok)) return rc;
    if (n_top > BPE_HEAD_MAX_TOP)
        return fail(ctx, BPE_ERR_INVALID_ARG, "head_logprobs: %u alternatives, at most %u", n_top, BPE_HEAD_MAX_TOP);
    if (n_rows == 0) return BPE_OK;
    if (d_logprob_out && !d_ids) return fail(ctx, BPE_ERR_INVALID_ARG, "head_logprobs: log-probabilities without ids");
    if (const int rc = head_report(ctx)) return rc;
    BPE_CUDA(ctx, cudaSetDevice(ctx->device), "cudaSetDevice");
    const ScoreParams P{{d_logits, stride, n_tok, temperature, d_temperature}, d_ids, n_top, d_logprob_out, d_entropy_out,
                        d_top_ids_out, d_top_logprob_out, d_norm_out};
    return type == BPE_F32    ? launch_logprobs<float>(ctx, P, n_rows)
           : type == BPE_BF16 ? launch_logprobs<__nv_bfloat16>(ctx, P, n_rows)
                              : launch_logprobs<__half>(ctx, P, n_rows);
}

extern "C" int head_logprobs_backward(bpe_ctx *ctx, const void *d_logits, uint64_t stride, int type, uint32_t n_rows,
                                      uint32_t n_tok, const int32_t *d_ids, float temperature, const float *d_temperature,
                                      const float *d_norm, const float *d_grad_logprob, const float *d_entropy,
                                      const float *d_grad_entropy, void *d_grad_out, uint64_t grad_stride) {
    if (!ctx) return BPE_ERR_INVALID_ARG;
    const char *const name = "head_logprobs_backward";
    if (const int rc = head_row_check(ctx, name, d_logits, stride, type, n_rows, n_tok)) return rc;
    if (const int rc = head_grad_check(ctx, name, d_logits, stride, type, n_rows, n_tok, d_grad_out, grad_stride)) return rc;
    if (n_rows == 0) return BPE_OK;
    if (!d_norm) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: null pointer", name);
    if (d_grad_logprob && !d_ids) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: a gradient of log-probabilities without ids", name);
    if (d_grad_entropy && !d_entropy) return fail(ctx, BPE_ERR_INVALID_ARG, "%s: a gradient of entropies without them", name);
    BPE_CUDA(ctx, cudaSetDevice(ctx->device), "cudaSetDevice");
    const ScoreGradParams P{{d_logits, stride, n_tok, temperature, d_temperature}, d_ids, d_norm, d_grad_logprob,
                            d_entropy, d_grad_entropy, d_grad_out, grad_stride};
    return type == BPE_F32    ? launch_backward<float>(ctx, P, n_rows)
           : type == BPE_BF16 ? launch_backward<__nv_bfloat16>(ctx, P, n_rows)
                              : launch_backward<__half>(ctx, P, n_rows);
}
