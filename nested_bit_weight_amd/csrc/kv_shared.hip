// kv_shared.hip -- attention of each row's new tokens over its cached slots, where
// groups of rows share a prefix that is read once for all of them, gfx950.
//
// For a line, a query head of a new token, with the n slots that the token sees
//     s_j = scale q.k_j,   o = sum_j 2^(s_j' - m) v_j / sum_j 2^(s_j' - m),
// s' = s log2(e), with any m near the largest s'.  Slots are cut in segments: a group's
// prefix (in the pages of its first row that has all of it), with all lines of the group, and each row's own slots behind it, with the row's
// lines.  What a segment gives a line, (m, sum, o), is joined in a last launch.
//
// Three launches.  The first divides the work: blocks of lines of a head (32, or 128 where segments have more) times runs
// of 128 slots, in equal shares over as many workgroups as run at once, whatever the lengths; so nothing but the
// device's own numbers says how long a row is, and a captured call stays valid as rows grow.  The second
// attends, prefixes and own slots side by side; the third joins the parts of each line.
//
// Few lines are bound by the cache's bytes: each of a workgroup's four waves has 32 of each 128 slots to itself, in LDS of its
// own, and never waits for the others until a piece ends.  Many lines are bound by the matrix units and the
// exponentials: each wave has 32 of the 128 lines, and the four share each tile's keys and values,
// so that LDS is read once for 32 lines but filled once for 128.
//
// Keys and values of bf16 go from memory straight to LDS, 16 bytes a lane, a tile (few lines: half a tile) ahead of their
// use; 8-bit ones through registers, widened to bf16, which holds them exactly.  The place of each 16-byte piece within a
// row is turned by the row's number so that readers do not meet in a bank.  Then on
// v_mfma_f32_32x32x16_bf16, with a line in each lane throughout:
//  - S^T = K Q^T: lane l has line l % 32 and of 32 slots the ones 8 (i / 4) + 4 (l / 32) + i % 4
//    in its registers i = 0..15, so the maximum and the sum need one exchange, between the halves;
//  - O^T = V^T P^T: these are the slots of P^T that the lane has to supply, if the product's inner
//    index 8 (l / 32) + j of step u stands for register 8 u + j; V^T comes from LDS by
//    transposing loads of four slots each, and o has its line in the lane too: rescaling it
//    is a product with the lane's own number.
//
// The weights enter the second product with all their 24 bits, as three bf16 parts, where lines are few; as they are then bound
// by bytes that costs little (16 rows of 4096 slots with 5 tokens 42.5 -> 43.5 us a call, 64 rows behind a prefix 49.3 -> 50.6).
// Many lines are bound by that product, and there the weights are rounded to bf16, half a step of 2^-8, unless the caller asks
// for all bits; the sum is then taken over the rounded ones, so that an average of equal values is exact and the error is that of
// the weights' differences, about as much again as the result's own rounding.  (Two parts, 16 bits, in blocks of 128 lines: 96 rows with 5 tokens
// behind a prefix of 32767 188 -> 253 us, 64 rows 49 -> 59; three: 320 and 66.)  With all bits asked for every block has 32 lines: 467 and 63.
//
// The running maximum m of a line is only raised, and o and the sum rescaled, when a score
// passes it by more than 8 (a factor of 2^8).
//
// Measured (32 query heads over 8 of 128 dims, bf16; the second launch as a trace's median, then a call's three): 64 rows behind a
// prefix of 8192, 600 slots of their own each, 122 MB: 39 (3.1 TB/s) and 50 us; 16 rows of 4096 slots with 5 tokens, 148 MB: 34
// us (4.3 TB/s) and 44; 96 rows with up to 5 tokens, 232 in all, behind a prefix of 32767, 125.5 GFLOP: 220 us (least 194; matrix units
// busy 38% of the time, VALU 35) and 205 without the trace, 610 TFLOP/s.  Loads through registers and barriers, prefixes and
// own slots in launches of their own: 148 us, 87 and 295 in all.
#include <algorithm>
#include <type_traits>

#include "kv.h"

namespace nbw {

typedef float f32x4_sh __attribute__((ext_vector_type(4)));
typedef float f32x16_sh __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2_sh __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8_sh __attribute__((ext_vector_type(8)));
typedef short i16x4_sh __attribute__((ext_vector_type(4)));

constexpr int SHARED_WAVES = 4;
constexpr int SHARED_THREADS = 64 * SHARED_WAVES;
constexpr int UNIT = 128;    // slots of a unit of work
constexpr float RAISE = 8.f; // how far a score may pass the running maximum

#define NEG_INF (-__builtin_inff())

// Lines and slots of a segment, as the first launch leaves them.
struct Segment {
    int row;             // whose table holds its slots
    int token, tokens;   // its lines' tokens
    int start, end;      // its slots
    int blocks;          // of lines, of a head
    int ranges, reach;   // pieces that the units of a block are cut into, and units of one
};
__device__ __forceinline__ int units_of(const Segment &s) { return (s.end - s.start + UNIT - 1) / UNIT; }  // of a block

// The call's division of work and its scratch.
struct SharedPlan {
    int group;                   // query heads of a head
    int wgs;                     // workgroups of the launch that attends
    int2 *tokens;                // [tokens] the token's row, or -1, and that row's group, or -1
    int32_t *sees;               // [tokens] slots that it sees
    struct Division {
        int32_t shares[2];       // of the workgroups, those of each side
        int32_t whole[2];        // whether shares end between pieces
    } *division;
    struct Side {                // 0: the groups' prefixes, 1: the rows' own slots
        int lines, segments;     // lines of a block, a power of two
        uint32_t places;         // that there are
        Segment *segment;        // [segments]
        uint32_t *cost;          // [segments + 1] of the segments before each
        uint32_t *parts;         // [segments] places of parts before each segment's
        float *ml, *o;           // [place][2] and [place][dim]: a line's part, its m and sum, and o.  First the
                                 // [wgs][lines] that a workgroup begins within a piece, then a place for
                                 // each piece's beginning: by segment, head, range and line
    } side[2];
};

// A piece costs as much as its units and START more, for the loads that depend on each other at its
// start and the result at its end (few lines: 7 us beside 3 for a unit; many: 8 beside 5).
constexpr int START = 2;
// Units that a share which ends within a piece costs beyond that, for what it writes and the join reads; and units that the
// join takes for each line that whole pieces would spare it (0.23 ns each, beside units of 5 and 3 us).  Calls divided and with
// whole pieces of own slots: 13 rows of up to 496 new tokens, 50 query heads over 10, 149 and 94 us (whole is taken); 61 rows of up to 27 49 and 40
// (whole); 64 rows behind a prefix of 8192 50 and 56, 16 rows of 4096 slots with 5 tokens 44 and 64 (divided).  34 rows of up to 395 new tokens behind
// 2000 slots of their own are divided, as their pieces would be longer than a share: 355 us, where whole ones take 288.
constexpr float CUT = 2.f;
constexpr float JOINED_MANY = 1.f / 22000, JOINED_FEW = 1.f / 13000;
__device__ __forceinline__ uint32_t head_cost(const Segment &s) {
    return (uint32_t)s.blocks * (uint32_t)(units_of(s) + START * s.ranges);
}

// All of a call's units, costs and places are below 2^31 (shared_plan); sums that say otherwise, of rows that are not
// what they should be, stay there.
constexpr uint32_t MOST = 0x7FFFFFFFu;
__device__ __forceinline__ uint32_t plus(uint32_t a, uint32_t b) { return min(a + b, MOST); }  // of two up to MOST
__device__ __forceinline__ uint32_t bounded(uint64_t x) { return (uint32_t)min(x, (uint64_t)MOST); }

// a * b / c, rounded down, of a below 2^31, b below 2^20 and c not 0: in fp64 exact, as no quotient is closer to the next
// whole number than 1 / c.  (A 64-bit division takes some 200 instructions.)
__device__ __forceinline__ uint32_t share_of(uint32_t a, uint32_t b, uint32_t c, double less = 0.0) {
    return (uint32_t)(((double)a * b - less) / c);
}

// A row's later blocks see more slots than its earlier ones, so they are taken in turn from its beginning and its end.
__device__ __forceinline__ int block_of(int nth, int blocks) { return nth & 1 ? blocks - 1 - nth / 2 : nth / 2; }
__device__ __forceinline__ int nth_of(int block, int blocks) { return block < (blocks + 1) / 2 ? 2 * block : 2 * (blocks - 1 - block) + 1; }

__device__ __forceinline__ int bounded(int x, int low, int high) { return min(max(x, low), high); }
__device__ __forceinline__ int first_token(const KvAttendShared &a, int row) {
    return a.cu ? bounded(a.cu[row], 0, a.tokens) : row;
}

// Entries 1 .. n of an ascending array, the ends of n runs that begin at entry 0: every stride-th of them in LDS, so
// that a search waits for memory only within a stride.
constexpr int PLAN_THREADS = 256;
constexpr int ENDS = 1024;
struct Ends {
    const int32_t *runs;
    int n, stride, kept;
    int32_t *s_ends;
    __device__ __forceinline__ void keep(const int32_t *r, int count, int32_t *lds) {
        runs = r;
        n = r ? count : 0;
        stride = max((n + ENDS - 1) / ENDS, 1);
        kept = (n + stride - 1) / stride;
        s_ends = lds;
        for (int i = threadIdx.x; i < kept; i += PLAN_THREADS) s_ends[i] = runs[min((i + 1) * stride, n)];
    }
    // The run that x is in, or -1.
    __device__ __forceinline__ int find(int x) const {
        int low = 0, high = kept;  // the first kept end past x
        while (low < high) {
            const int mid = (low + high) / 2;
            if (s_ends[mid] <= x) low = mid + 1;
            else high = mid;
        }
        if (low == kept) return -1;
        low *= stride;
        high = min(low + stride, n) - 1;
        while (low < high) {
            const int mid = (low + high) / 2;
            if (runs[mid + 1] <= x) low = mid + 1;
            else high = mid;
        }
        return runs[low] <= x ? low : -1;
    }
};

constexpr int N_SUMS = 5;  // at a time

// The sums of N numbers over the workgroup's threads up to this one, in x, and over all.
template <int N, int THREADS>
__device__ __forceinline__ void add_up(uint32_t (&x)[N], uint32_t (&all)[N], uint32_t (*s_wave)[N_SUMS]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = (uint32_t)wave_running((int32_t)x[i], 0, [](int32_t a, int32_t b) { return (int32_t)plus((uint32_t)a, (uint32_t)b); });
    if (lane == 63)
#pragma unroll
        for (int i = 0; i < N; ++i) s_wave[wave][i] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        all[i] = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) {
            if (w < wave) x[i] = plus(x[i], s_wave[w][i]);
            all[i] = plus(all[i], s_wave[w][i]);
        }
    }
    __syncthreads();
}

// The last workgroup of the launch divides the work, the others find each token's row.
__global__ __launch_bounds__(PLAN_THREADS) void kv_shared_plan_kernel(KvCache c, KvAttendShared a, SharedPlan pl) {
    __shared__ uint32_t s_wave[PLAN_THREADS / 64][N_SUMS];
    __shared__ int32_t s_ends[2][ENDS];
    __shared__ int s_longest[PLAN_THREADS / 64];
    const int tid = threadIdx.x;
    Ends groups, rows;
    groups.keep(a.group_rows, a.groups, s_ends[0]);
    if (blockIdx.x + 1 < gridDim.x) {
        rows.keep(a.cu, c.rows, s_ends[1]);
        __syncthreads();
        const int token = blockIdx.x * PLAN_THREADS + tid;
        if (token >= a.tokens) return;
        int row = token, behind = 0;
        if (a.cu) {
            row = rows.find(token);
            if (row >= 0) behind = min(a.cu[row + 1], a.tokens) - 1 - token;
        }
        pl.tokens[token] = int2{row, row < 0 ? -1 : groups.find(row)};
        pl.sees[token] = row < 0 ? 0 : max(kv_len(a.lens, row, a.max_len) - behind, 0);
        return;
    }
    __syncthreads();
    // A strip of segments for each thread; with no more segments than threads its one stays in registers.
    auto alone = [&](int g) { return a.group_rows[g + 1] - a.group_rows[g] == 1; };  // one row shares with no other
    // A group's lines and slots.  Its prefix is read through the table of its first row that is as long as the prefix, else of
    // the longest one and as far as that has it.  (What a shorter row's table says there may be another row's.)  A thread looks at
    // its group's first rows, as a rule at one; longer runs are looked at by the wave, which takes all of its lanes' groups.
    auto group = [&](int s) {
        Segment x = {0, 0, 0, 0, 0, 0, 0, 1};
        int r = 0, r1 = 0, prefix = 0, len = 0, best = -1;
        if (s < pl.side[0].segments && !alone(s)) {
            x.row = r = bounded(a.group_rows[s], 0, c.rows);
            r1 = bounded(a.group_rows[s + 1], 0, c.rows);
            prefix = bounded(a.prefix[s], 0, a.max_len);
            len = kv_len(a.lens, min(r, c.rows - 1), a.max_len);
            x.token = first_token(a, r);
            x.tokens = max(first_token(a, max(r, r1)) - x.token, 0);
        }
        auto look = [&](int at, int n) {
            if (n > best) {
                best = n;
                x.row = at;
            }
        };
        for (const int few = min(r + 4, r1); r < few && best < prefix;) {
            look(r, len);
            if (++r < few) len = kv_len(a.lens, r, a.max_len);
        }
        for (unsigned long long left = __ballot(r < r1 && best < prefix); left; left &= left - 1) {
            const int src = __builtin_ctzll(left), end = __builtin_amdgcn_readlane(r1, src), enough = __builtin_amdgcn_readlane(prefix, src);
            int at = __builtin_amdgcn_readlane(r, src), top = __builtin_amdgcn_readlane(best, src), top_row = -1;
            for (; at < end && top < enough; at += 64) {
                const int mine = at + (tid & 63), n = mine < end ? min(kv_len(a.lens, mine, a.max_len), enough) : -1, most = wave_max(n);
                if (most > top) {
                    top = most;
                    top_row = at + __builtin_ctzll(__ballot(n == most));
                }
            }
            if ((tid & 63) == src && top_row >= 0) look(top_row, top);
        }
        x.end = bounded(best, 0, prefix);
        return x;
    };
    auto of = [&](int which, int s, Segment group) {
        Segment x = {s, 0, 0, 0, 0, 0, 0, 1};
        if (!which) {
            x = group;
        } else {
            const int t0 = first_token(a, s), t1 = first_token(a, s + 1), g = groups.find(s);
            x.token = t0;
            x.tokens = max(t1 - t0, 0);
            x.start = g < 0 || alone(g) ? 0 : bounded(a.prefix[g], 0, a.max_len);
            x.end = kv_len(a.lens, s, a.max_len);
        }
        if (x.tokens == 0) x.end = x.start;
        x.end = max(x.end, x.start);
        x.blocks = units_of(x) ? (int)(((int64_t)x.tokens * pl.group + pl.side[which].lines - 1) >> __builtin_ctz(pl.side[which].lines)) : 0;
        return x;
    };
    int s0[2], s1[2];
    Segment mine[2];
    {
        const int n = pl.side[0].segments, strip = (n + PLAN_THREADS - 1) / PLAN_THREADS;
        for (int i = 0; i < strip; ++i) {  // in all lanes
            mine[0] = group(tid * strip + i);
            if (strip > 1 && tid * strip + i < n) pl.side[0].segment[tid * strip + i] = mine[0];
        }
    }
    auto kept = [&](int which, int s, bool one) {  // what group() gave
        if (which || one) return mine[0];
        return pl.side[0].segment[s];
    };
    int own_units = 0;  // the most of a row's own slots
    uint32_t sums[5] = {0, 0, 0, 0, 0}, all[5];  // units and blocks of both sides, and tokens that see no prefix
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const int n = pl.side[which].segments, strip = (n + PLAN_THREADS - 1) / PLAN_THREADS;
        s0[which] = min(tid * strip, n);
        s1[which] = min(s0[which] + strip, n);
        for (int s = s0[which]; s < s1[which]; ++s) {
            const Segment x = mine[which] = of(which, s, kept(which, s, strip == 1));
            const uint32_t blocks = bounded((uint64_t)c.heads * x.blocks);
            sums[which] = plus(sums[which], bounded((uint64_t)blocks * units_of(x)));
            sums[2 + which] = plus(sums[2 + which], blocks);
            if (which) own_units = max(own_units, units_of(x));
            if (which && x.start == 0) sums[4] = plus(sums[4], (uint32_t)x.tokens);
        }
    }
    own_units = wave_max(own_units);
    if ((tid & 63) == 0) s_longest[tid >> 6] = own_units;
    add_up<5, PLAN_THREADS>(sums, all, s_wave);
    int longest = 0;
#pragma unroll
    for (int w = 0; w < PLAN_THREADS / 64; ++w) longest = max(longest, s_longest[w]);
    // Workgroups by the sides' cost, a unit of many lines taking 5/4 of the time of one of few; one for each
    // unit at the most, and one for a side that has any.
    uint32_t shares[2] = {all[0], all[1]};
    if (plus(all[0], all[1]) > (uint32_t)pl.wgs) {
        const double w0 = ((double)all[0] + START * (double)all[2]) * (pl.side[0].lines > 32 ? 5 : 4);
        const double w1 = ((double)all[1] + START * (double)all[3]) * (pl.side[1].lines > 32 ? 5 : 4);
        const uint32_t n0 = (uint32_t)(pl.wgs * w0 / (w0 + w1) + 0.5);
        shares[0] = min(min(max(n0, (uint32_t)(w0 > 0)), (uint32_t)pl.wgs - (w1 > 0)), all[0]);
        shares[1] = min(pl.wgs - shares[0], all[1]);
    }
    // A piece has no more units than an equal share: the blocks of a range of slots then go to
    // neighbouring workgroups, which meet its keys and values at about the same time.  Of rows' own slots the
    // shares may be of whole blocks: they differ by up to a block, but none that sees nothing else
    // has to be joined, and no piece is begun twice.
    int reach[2] = {shares[0] ? (int)((all[0] - 1) / shares[0] + 1) : 1, shares[1] ? (int)((all[1] - 1) / shares[1] + 1) : 1};
    const float shares1 = (float)max(shares[1], 1u), piece = (float)(longest + START);
    const float takes = all[3] <= shares[1] ? piece : ((float)all[1] + START * (float)all[3]) / shares1 + piece;
    const float divided = ((float)all[1] + START * ((float)all[3] + 0.5f * shares1)) / shares1 + START + CUT +
                      (float)all[4] * pl.group * c.heads * (pl.side[1].lines > 32 ? JOINED_MANY : JOINED_FEW);
    const int whole[2] = {0, longest <= reach[1] || all[3] <= shares[1] ? takes < divided : 0};
    if (whole[1]) reach[1] = max(reach[1], longest);
    auto cut = [&](int which, Segment &x) {
        x.ranges = units_of(x) ? (units_of(x) - 1) / reach[which] + 1 : 0;
        x.reach = x.ranges ? (units_of(x) - 1) / x.ranges + 1 : 1;
    };
    auto places_of = [&](const Segment &x) { return bounded((uint64_t)x.ranges * c.heads * ((uint64_t)x.tokens * pl.group)); };
    auto cost_of = [&](const Segment &x) { return bounded((uint64_t)c.heads * x.blocks * (uint64_t)(units_of(x) + START * x.ranges)); };
    uint32_t next[4] = {0, 0, 0, 0}, next_all[4];  // places and costs of both sides
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        if (tid == 0) {
            pl.division->whole[which] = whole[which];
            pl.division->shares[which] = (int)shares[which];
        }
        const bool one = s1[which] - s0[which] <= 1;
        for (int s = s0[which]; s < s1[which]; ++s) {
            if (!one) mine[which] = of(which, s, kept(which, s, false));
            cut(which, mine[which]);
            next[which] = plus(next[which], places_of(mine[which]));
            next[2 + which] = plus(next[2 + which], cost_of(mine[which]));
        }
    }
    const uint32_t own[4] = {next[0], next[1], next[2], next[3]};
    add_up<4, PLAN_THREADS>(next, next_all, s_wave);
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const auto &side = pl.side[which];
        uint32_t place = next[which] - own[which], cost = next[2 + which] - own[2 + which];
        const bool one = s1[which] - s0[which] <= 1;
        for (int s = s0[which]; s < s1[which]; ++s) {
            if (!one) {
                mine[which] = of(which, s, kept(which, s, false));
                cut(which, mine[which]);
            }
            Segment x = mine[which];
            side.parts[s] = place;
            side.cost[s] = cost;
            place = plus(place, places_of(x));
            cost = plus(cost, cost_of(x));
            // Rows that say they have the same tokens would need more places than there are: no lines then.
            if (plus(place, (uint32_t)(pl.wgs * side.lines)) > side.places) x.tokens = 0;
            side.segment[s] = x;
        }
        if (tid == 0) side.cost[side.segments] = next_all[2 + which];
    }
}

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
    const bf16x2_sh p = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, p);
}
template <int HALF>
__device__ __forceinline__ uint32_t fp8_widened(uint32_t w) {  // two 8-bit values of a word as bf16, exact
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HALF));
}
__device__ __forceinline__ u32x2_kv transposed(const uint8_t *lds) {
    return __builtin_bit_cast(u32x2_kv, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4_sh *)lds));
}

// What follows from these numbers is worked out again from here on, not kept ready in registers
// from before the loop: there are none to spare.
template <class... T>
__device__ __forceinline__ void again(T &...x) {
    (..., ([](auto &y) { asm volatile("" : "+v"(y)); })(x));
}
__device__ __forceinline__ float rounded_product(float a, float b) {  // by itself, not as part of a sum
#pragma clang fp contract(off)
    return a * b;
}
template <int LOADS_LEFT>
__device__ __forceinline__ void wait_loads() {  // all but the last so many have arrived; nothing is moved across
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(LOADS_LEFT) : "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void wait_lds() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}
__device__ __forceinline__ void meet() {  // the workgroup's waves, their LDS accesses done
    wait_lds();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
}

// Nothing is moved across: what is written before it is asked for, or begun, before what follows.
__device__ __forceinline__ void in_order() { __builtin_amdgcn_sched_barrier(0); }

// How a workgroup takes its lines.  Few: 32, and of each 128 slots a wave has 32, in LDS of its
// own, so that no wave waits for another.  Many: 128, 32 to a wave, over tiles in two buffers
// that the waves fill together.
template <int DIM, bool FP8, bool FEW>
struct Shape {
    static constexpr int LINES = FEW ? 32 : 32 * SHARED_WAVES;
    // Runs of 32 slots that a wave takes at once: two would leave no registers for 8-bit values on their way, or for 256 dims.
    static constexpr int SUBS = !FEW && DIM < (FP8 ? 128 : 256) ? 2 : 1;
    static constexpr int TILE = 32 * SUBS;                       // slots in LDS, of a wave, or of all
    static constexpr int STEP = FEW ? TILE * SHARED_WAVES : TILE; // slots from one of a wave's tiles to the next
    static constexpr int PIECES = DIM / 8;                       // of a slot's row, 16 bytes each
    static constexpr int ROWS = 64 / PIECES;                     // that a wave's lanes have a piece each of
    static constexpr int FILLED = FEW ? TILE : TILE / SHARED_WAVES; // rows of a tile that a wave fills
    static constexpr int LOADS = FILLED / ROWS;                  // of a lane for them, of keys and of values
    static constexpr int ROW = DIM * 2;
    static constexpr int PART = 32 * (DIM + 4) * 4;              // a wave's o, its rows 16 bytes past the banks' turn
    static constexpr int OWN = std::max(2 * TILE * ROW, PART);   // of a wave
    static constexpr int TILES = FEW ? OWN * SHARED_WAVES : 4 * TILE * ROW;
    // Queries of 256 dims would take 64 registers; each lane has its part of them in LDS instead.  (Waves with the same
    // lines write the same there.)
    static constexpr bool Q_LDS = DIM > 128;
    static constexpr int BYTES = TILES + (Q_LDS ? LINES * ROW : 0);
};

// 16 bytes of each lane to LDS, side by side from `lds` on, which is the same for all of them.  Written out, as the
// compiler puts a wait for all such loads before each transposing read, whatever that reads; what
// has to have arrived is said by wait_loads.
__device__ __forceinline__ void load_to_lds(const uint8_t *p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(lds) : "memory", "m0");
}

struct SharedLds {
    uint8_t *pool;
    float (*m)[32], (*l)[32];   // by wave and line
};

// One workgroup's share of a side's units.
template <int DIM, bool FP8, bool FEW>
__device__ __forceinline__ void attend_share(const KvCache &c, const KvAttendShared &a, const SharedPlan &pl, int which, int share,
                                             int shares, bool whole, const SharedLds &lds) {
    using X = Shape<DIM, FP8, FEW>;
    constexpr int TILE = X::TILE, SUBS = X::SUBS, PIECES = X::PIECES, LOADS = X::LOADS, ROW = X::ROW;
    constexpr int R = 256 / DIM;  // rows of a tile in 512 bytes, one turn of the banks
    constexpr int DB = DIM / 32, QF = DIM / 16;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = lane >> 5, col = lane & 31;
    const auto &side = pl.side[which];
    const uint32_t all_cost = side.cost[side.segments];
    uint32_t u = share_of(all_cost, share, shares);
    const uint32_t u1 = share_of(all_cost, share + 1, shares);
    int seg = 0;  // segments that end at or before u: 64 places looked at together, then 64 between two of them
    for (int high = side.segments; seg < high;) {
        const int step = (high - seg + 63) / 64, at = seg + (lane + 1) * step;
        seg += step * __popcll(__ballot(at <= high && side.cost[at] <= u));
        high = min(seg + step - 1, high);
    }

    // A row of a tile has its pieces at places turned by the row's number s.  Keys, whose readers have 32 rows side by
    // side, 16 bytes each: by (s / R) % PIECES.  Values, whose readers have 8 rows and 64 bytes of each: by 4 v_way(s),
    // which puts rows 0..3, 4..7, the even and the odd ones each in banks of their own.  A lane fills place
    // l % PIECES of rows ROWS i + l / PIECES (from a multiple of 8 on), of which s / R is 2 i + l / 32, and v_way that
    // of l / PIECES turned by bits of i: so the piece it loads for i differs from that for 0 by bits of i.
    auto v_way = [](int s) { return DIM == 64 ? (s >> 1 ^ s >> 2) & 1 : DIM == 128 ? (s & 3) ^ (s >> 2 & 1) : s & 7; };
    const int first_row = FEW ? 0 : wave * X::FILLED;  // that the wave fills
    const int fill_row = lane / PIECES;
    const int k_fill = (lane % PIECES) ^ ((first_row / R + half) & (PIECES - 1));
    const int v_fill = (lane % PIECES) ^ (v_way(fill_row) << 2);
    const int k_read = col * ROW, k_turn = (half ^ ((col / R) & (PIECES - 1))) << 4;
    const int v_slot = 4 * half + (lane & 15) / 4;
    const int v_turn = v_way(v_slot) << 6;
    const int v_read = v_slot * ROW + (2 * ((lane >> 4) & 1) + (lane & 3) / 2) * 16 + (lane & 1) * 8;
    uint8_t *const own = lds.pool + (FEW ? wave * X::OWN : 0);
    const uint32_t own_at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) void *)own);

    auto next_segment = [&] {  // past the ones without work
        for (int n = 64; n == 64; seg += n)
            n = __popcll(__ballot(seg + lane < side.segments && side.cost[seg + lane + 1] <= u));
    };
    // The piece that u is in: `nth` of the blocks of a head's range, whose pieces have `len` units, and how far in.
    struct Piece {
        int head, range, reach, len, nth, off;
    };
    auto piece_at = [&](const Segment &sg) {
        const int reach = sg.reach;
        const uint32_t in = u - side.cost[seg], per_head = head_cost(sg), per_range = (uint32_t)sg.blocks * (uint32_t)(reach + START);
        const int head = (int)(in / per_head);
        const uint32_t in_head = in - head * per_head;
        const int range = min((int)(in_head / per_range), sg.ranges - 1);
        const uint32_t in_range = in_head - range * per_range;
        const int len = min(reach, units_of(sg) - range * reach);
        const int nth = (int)(in_range / (uint32_t)(len + START));
        return Piece{head, range, reach, len, nth, (int)in_range - nth * (len + START)};
    };
    if (whole) {  // a piece that the share before has begun is its own
        const Piece p = piece_at(side.segment[seg]);
        if (p.off) u += p.len + START - p.off;
        if (u >= u1) return;
        next_segment();
    }
    for (;;) {  // a piece, or a part of one: units [c0, c1) of one block of a segment's lines
        const Segment sg = side.segment[seg];
        const auto [head, range, reach, len, nth, off] = piece_at(sg);
        const int rest = len + START - off, take = whole ? rest : (int)min(u1 - u, (uint32_t)rest);
        const int block = which ? block_of(nth, sg.blocks) : nth;
        const int c0 = range * reach + max(off - START, 0), c1 = range * reach + max(off + take - START, 0);
        const bool begins = off <= START;
        u += take;
        if (c0 == c1) return;  // the share ends before the piece's first unit
        if (sg.tokens == 0) return;
        const int nlines = min(X::LINES, sg.tokens * pl.group - block * X::LINES);
        const int from = sg.start + c0 * UNIT + (FEW ? wave * TILE : 0);  // the wave's first slot
        const int32_t *table = c.table + (int64_t)sg.row * c.table_ld;

        // 64 pages of the table from pages_at on, one in each lane, as the number of the pool's row that the head's slots
        // begin with there; and which of them are not there (the pool's first page is read in their place).
        uint32_t pages;
        uint64_t gone = 0;
        int pages_at;
        auto ask_pages = [&](int slot) {
            pages_at = min(slot, c.cap - 1) >> c.page_log2;
            const int32_t page = table[min(pages_at + lane, c.width - 1)];
            const bool there = page >= 0 && page < c.pages;
            gone = __ballot(!there);
            pages = ((uint32_t)(there ? page : 0) * (uint32_t)c.heads + (uint32_t)head) << c.page_log2;
        };
        ask_pages(from);

        const int line = FEW ? col : wave * 32 + col;
        const bool valid = line < nlines;
        const int seg_line = block * X::LINES + (valid ? line : 0);
        const int token = sg.token + seg_line / pl.group, q_head = head * pl.group + seg_line % pl.group;
        u32x4_kv q[X::Q_LDS ? 1 : QF];
        uint8_t *const q_own = lds.pool + X::TILES + (FEW ? 0 : wave * 32 * ROW) + k_read;
        {
            const uint16_t *src = a.q + (int64_t)token * a.q_ld + (int64_t)q_head * DIM + half * 8;
            const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
            for (int f = 0; f < QF; ++f) {
                u32x4_kv x = *reinterpret_cast<const u32x4_kv *>(src + f * 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = valid ? x[e] ^ flip : 0u;
                if constexpr (X::Q_LDS) *reinterpret_cast<u32x4_kv *>(q_own + (k_turn ^ (f << 5))) = x;
                else q[f] = x;
            }
        }
        // The last slot that any line sees: a row's later tokens see more.
        const int end = which ? min(sg.end, pl.sees[sg.token + (block * X::LINES + nlines - 1) / pl.group]) : sg.end;
        const int to = min(sg.start + c1 * UNIT, end);
        const int tiles = to > from ? (to - from + X::STEP - 1) / X::STEP : 0;
        const int sees = valid ? min(pl.sees[token], to) : INT32_MAX;
        const int least = -wave_max(-sees), most = wave_max(valid ? sees : 0);
        // (Not 0, which an infinite score would make a NaN of: what is smaller tells no two finite scores apart.)
        const float by = fmaxf(fabsf(a.scale) * 1.44269504088896340736f * (FP8 ? c.k_scale[head] : 1.f), 0x1p-126f);
        // Weights are up to 2^RAISE, and as many meet the values as the segment has slots: times a
        // power of two, in their exponent, they sum to 1 at the most, and finite values cannot run over (but for scores so large,
        // past 2^27, that nothing can be taken off them).
        const int n = sg.end - sg.start;
        const float room = RAISE + (n > 1 ? 32 - __builtin_clz(n - 1) : 0);

        // Where a tile's slots are: for each row that this lane loads a piece of, its place in a pool counted in pieces.
        // Tells whether a slot's page is not there.
        uint32_t rows[LOADS];
        auto find = [&](int tile) {
            const int slot0 = min(from + tile * X::STEP, c.cap - 1), slot1 = min(slot0 + TILE, c.cap) - 1;
            if ((slot1 >> c.page_log2) - pages_at >= 64) ask_pages(slot0);
            const int at0 = (slot0 >> c.page_log2) - pages_at, at1 = (slot1 >> c.page_log2) - pages_at;
            const int slot = min(slot0 + lane % TILE, slot1);
            const uint32_t mine = (__shfl(pages, (slot >> c.page_log2) - pages_at) + (slot & ((1 << c.page_log2) - 1))) * PIECES;
            int row = first_row + fill_row;
            again(row);
#pragma unroll
            for (int i = 0; i < LOADS; ++i) rows[i] = __shfl(mine, row + i * X::ROWS);
            return (gone << (63 - at1) >> (63 - at1 + at0)) != 0;
        };
        // 8-bit values come through registers, to be widened.
        u32x2_kv raw[FP8 ? 2 : 1][LOADS];
        auto load = [&](bool values, int to_own) {
            int fill = values ? v_fill : k_fill;
            again(fill);
            const uint8_t *pool = values ? c.v : c.k;
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const uint64_t at = rows[i] + (uint32_t)(values ? fill ^ (v_way(i * X::ROWS) << 2) : fill ^ 2 * i);
                if constexpr (FP8) raw[values][i] = *reinterpret_cast<const u32x2_kv *>(pool + (at << 3));
                else load_to_lds(pool + (at << 4), own_at + to_own + i * 1024);
            }
        };
        auto widen = [&](bool values, int to_own) {
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < LOADS; ++i) {
                    const u32x2_kv w = raw[values][i];
                    *reinterpret_cast<u32x4_kv *>(own + to_own + i * 1024 + lane * 16) =
                        u32x4_kv{fp8_widened<0>(w[0]), fp8_widened<1>(w[0]), fp8_widened<0>(w[1]), fp8_widened<1>(w[1])};
                }
            }
        };

        f32x16_sh o[DB];
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
        float m = NEG_INF, sum = 0.f;
        f32x16_sh s[SUBS];
        constexpr int PARTS = FEW ? 3 : 1;  // of a weight
        u32x4_kv p[SUBS][2][PARTS];

        // S^T of the tile whose keys are at kb; the keys AHEAD products on are under way.
        constexpr int AHEAD = 3;
        auto scores = [&](const uint8_t *kb) {
            int row = k_read, way = k_turn;
            again(row, way);
            constexpr int PRODUCTS = SUBS * QF;
            u32x4_kv kf[AHEAD + 1], qf[X::Q_LDS ? AHEAD + 1 : 1];
            auto ask = [&](int j) {
                kf[j % (AHEAD + 1)] = *reinterpret_cast<const u32x4_kv *>(kb + j / QF * 32 * ROW + row + (way ^ (j % QF << 5)));
                if constexpr (X::Q_LDS) qf[j % (AHEAD + 1)] = *reinterpret_cast<const u32x4_kv *>(q_own + (way ^ (j % QF << 5)));
            };
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) ask(j);
#pragma unroll
            for (int b = 0; b < SUBS; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
#pragma unroll
            for (int j = 0; j < PRODUCTS; ++j) {
                if (j + AHEAD < PRODUCTS) ask(j + AHEAD);
                in_order();
                const u32x4_kv &qj = X::Q_LDS ? qf[j % (AHEAD + 1)] : q[j % QF];
                s[j / QF] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_sh, kf[j % (AHEAD + 1)]),
                                                                    __builtin_bit_cast(bf16x8_sh, qj), s[j / QF], 0, 0, 0);
            }
        };
        // The running maximum, for the scores in s, which get their factor; gives what the weights are taken from.  `first` is the
        // tile's first slot, `all` says that every line sees the whole tile.  (The factor's product is rounded before anything is taken
        // from it, as the maximum is: of scores past 2^31 the two would differ by more than an exponential bears.  In one step, product
        // and difference take 200 us in place of 205 of the document, 152 of 156 at 256 dims, and as long within 1% elsewhere.)
        auto raise = [&](int first, auto all, const uint32_t *there) {
            if constexpr (!decltype(all)::value) {
#pragma unroll
                for (int b = 0; b < SUBS; ++b) {
                    const int left = sees - first - b * 32 - 4 * half;  // slots that the line sees, from the lane's first on
                    const uint32_t mine = there[b] >> (4 * half);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = 8 * (i / 4) + i % 4;
                        s[b][i] = (mine >> j & 1) && j < left ? s[b][i] : NEG_INF;
                    }
                }
            }
            float top = NEG_INF;
#pragma unroll
            for (int b = 0; b < SUBS; ++b)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    s[b][i] = rounded_product(s[b][i], by);
                    top = fmaxf(top, s[b][i]);
                }
            if (__any(top + room > m + RAISE)) {
                top = fmaxf(top, __shfl_xor(top, 32)) + room;
                top = fmaxf(m, top);
                const float fade = top == m ? 1.f : __builtin_amdgcn_exp2f(m - top);  // equal: -inf, or nothing to do
                m = top;
                sum *= fade;
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[d][i] *= fade;
            }
            return m == NEG_INF ? 0.f : m;
        };
        // Weights 2 i and 2 i + 1 of run b, in s in the scores' place, their bf16 parts in p, and in `part` the sum of what these stand for.
        auto weigh = [&](int b, int i, float ref, float &part) {
            s[b][2 * i] = __builtin_amdgcn_exp2f(s[b][2 * i] - ref);
            s[b][2 * i + 1] = __builtin_amdgcn_exp2f(s[b][2 * i + 1] - ref);
            auto &mine = p[b][i / 4];
            if constexpr (PARTS == 1) {
                const bf16x2_sh two = {(__bf16)s[b][2 * i], (__bf16)s[b][2 * i + 1]};
                part = __builtin_amdgcn_fdot2_f32_bf16(two, bf16x2_sh{(__bf16)1.f, (__bf16)1.f}, part, false);
                mine[0][i % 4] = __builtin_bit_cast(uint32_t, two);
            } else {
                // Each part but the last is cut off, not rounded, so that none is negative; and what is left is no less than
                // the smallest normal number, or than the weight itself: the middle one of the three.  So no part is
                // 0 unless the weight is, and an infinite value stays one.
                constexpr float TINY = 0x1p-126f;
                float w0 = s[b][2 * i], w1 = s[b][2 * i + 1];
                part += w0 + w1;
#pragma unroll
                for (int x = 0; x + 1 < PARTS; ++x) {
                    const uint32_t cut = __builtin_amdgcn_perm(__float_as_uint(w1), __float_as_uint(w0), 0x07060302u);
                    mine[x][i % 4] = cut;
                    w0 = __builtin_amdgcn_fmed3f(w0 - bf16_lo(cut), TINY, w0);
                    w1 = __builtin_amdgcn_fmed3f(w1 - bf16_hi(cut), TINY, w1);
                }
                mine[PARTS - 1][i % 4] = bf16_pair(w0, w1);
            }
        };
        // Adds 16 values, of some dims, times the weights of step k.
        auto add_step = [&](f32x16_sh &to, const u32x4_kv &values, int k) {
#pragma unroll
            for (int x = 0; x < PARTS; ++x)
                to = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_sh, values),
                                                             __builtin_bit_cast(bf16x8_sh, p[k / 2][k % 2][x]), to, 0, 0, 0);
        };
        // O^T with the values at vb.  Step k is 16 slots: while its products run, the values three products on are under
        // way and the next step's weights are worked out.
        auto add = [&](const uint8_t *vb, float ref) {
            int row = v_read, way = v_turn;
            again(row, way);
            constexpr int PRODUCTS = 2 * SUBS * DB;
            u32x4_kv vf[AHEAD + 1];
            auto ask = [&](int j) {
                const uint8_t *src = vb + 16 * (j / DB) * ROW + row + ((j % DB << 6) ^ way);
                const u32x2_kv v0 = transposed(src), v1 = transposed(src + 8 * ROW);
                vf[j % (AHEAD + 1)] = u32x4_kv{v0[0], v0[1], v1[0], v1[1]};
            };
            float part = 0.f;  // of a long sum, so that few roundings follow each other
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) ask(j);
            in_order();
#pragma unroll
            for (int i = 0; i < 4; ++i) weigh(0, i, ref, part);
#pragma unroll
            for (int j = 0; j < PRODUCTS; ++j) {
                const int k = j / DB, d = j % DB;
                if (j + AHEAD < PRODUCTS) ask(j + AHEAD);
                in_order();
                add_step(o[d], vf[j % (AHEAD + 1)], k);
                if (j + DB < PRODUCTS)
#pragma unroll
                    for (int i = d * 4 / DB; i < (d + 1) * 4 / DB; ++i) weigh((k + 1) / 2, (k + 1) % 2 * 4 + i, ref, part);
            }
            sum += part;
        };
        // The same where a slot may not count, for a line or for all: its weight is 0, but what
        // lies there may be NaN or infinite.  Such values are left out of the product and added to the
        // lines that do see them, one slot after the other.
        auto add_with_care = [&](const uint8_t *vb, int first, const uint32_t *there, float ref) {
            uint32_t odd[SUBS] = {};  // slots with such a value
            for (int i = 0; i < TILE / X::ROWS; ++i) {
                const u32x4_kv x = *reinterpret_cast<const u32x4_kv *>(vb + i * 1024 + lane * 16);
                bool any = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) any = any || (x[e] & 0x7F80u) == 0x7F80u || (x[e] & 0x7F800000u) == 0x7F800000u;
                const uint64_t lanes = __ballot(any);
                if (lanes)
#pragma unroll
                    for (int r = 0; r < X::ROWS; ++r)
                        if (lanes >> (r * PIECES) & (~0ull >> (64 - PIECES))) {
                            const int j = i * X::ROWS + r;
                            if (SUBS == 1 || j < 32) odd[0] |= 1u << (j & 31);
                            else odd[SUBS - 1] |= 1u << (j & 31);
                        }
            }
            bool any = false;
#pragma unroll
            for (int b = 0; b < SUBS; ++b) any = any || odd[b];
            if (!any) {
                add(vb, ref);
                return;
            }
            float part = 0.f;
            int row = v_read, way = v_turn;
            again(row, way);
#pragma unroll
            for (int k = 0; k < 2 * SUBS; ++k) {
#pragma unroll
                for (int i = 0; i < 4; ++i) weigh(k / 2, k % 2 * 4 + i, ref, part);
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    in_order();  // few loads at a time
                    const uint8_t *src = vb + 16 * k * ROW + row + ((d << 6) ^ way);
                    const u32x2_kv v0 = transposed(src), v1 = transposed(src + 8 * ROW);
                    u32x4_kv vf = {v0[0], v0[1], v1[0], v1[1]};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if ((vf[e] & 0x7F80u) == 0x7F80u) vf[e] &= 0xFFFF0000u;
                        if ((vf[e] & 0x7F800000u) == 0x7F800000u) vf[e] &= 0x0000FFFFu;
                    }
                    add_step(o[d], vf, k);
                }
            }
            sum += part;
            int dim0 = 4 * half;
            again(dim0);
#pragma unroll
            for (int b = 0; b < SUBS; ++b)
                for (uint32_t rest = odd[b] & there[b]; rest; rest &= rest - 1) {
                    const int j = __builtin_ctz(rest);
                    if (first + b * 32 + j >= most) break;
                    float w = 0.f;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (8 * (i / 4) + i % 4 == (j & ~4)) w = s[b][i];
                    w = __shfl(w, col + 32 * (j >> 2 & 1));
                    const bool seen = first + b * 32 + j < sees;
                    const int row = b * 32 + j, turn = v_way(row) << 6;
                    const uint8_t *src = vb + row * ROW + dim0 * 2;
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            if (i % 4 == 0) in_order();  // few loads at a time
                            const uint32_t x = *reinterpret_cast<const uint16_t *>(src + (((d << 6) ^ turn) + 16 * (i / 4) + 2 * (i % 4)));
                            if ((x & 0x7F80u) == 0x7F80u && seen) o[d][i] += w * __uint_as_float(x << 16);
                        }
                    }
                }
        };
        // Which slots of a tile are on pages that are there, where some are not.
        auto present = [&](int first, bool missing, uint32_t *there) {
#pragma unroll
            for (int b = 0; b < SUBS; ++b) {
                there[b] = ~0u;
                if (missing) {
                    const int32_t pg = table[min(first + b * 32 + col, c.cap - 1) >> c.page_log2];
                    there[b] = (uint32_t)__ballot(pg >= 0 && pg < c.pages);
                }
            }
        };

        if constexpr (FEW) {
            // Keys and values in turn: as soon as a tile's keys are used the next one's are asked for, and so
            // the values, so that one half or the other is always under way.
            constexpr int KEYS = 0, VALUES = TILE * ROW;
            const uint8_t *kb = own + KEYS, *vb = own + VALUES;
            bool missing = false;
            if (tiles > 0) {
                missing = find(0);
                load(false, KEYS);
                load(true, VALUES);
            }
            auto step = [&](int t, auto all) {
                const int first = from + t * X::STEP;
                if constexpr (FP8) widen(false, KEYS);
                else wait_loads<LOADS>();  // the values
                scores(kb);
                wait_lds();
                uint32_t there[SUBS];
                if constexpr (!decltype(all)::value) present(first, missing, there);
                missing = find(min(t + 1, tiles - 1));
                if constexpr (FP8) widen(true, VALUES);
                load(false, KEYS);
                const float ref = raise(first, all, there);
                if constexpr (!FP8) wait_loads<LOADS>();  // the next keys
                if constexpr (decltype(all)::value) add(vb, ref);
                else add_with_care(vb, first, there, ref);
                wait_lds();
                load(true, VALUES);
            };
            int t = 0;
            for (; t < tiles && from + t * X::STEP + TILE <= least && !missing; ++t) step(t, std::true_type());
            for (; t < tiles; ++t) step(t, std::false_type());
            if constexpr (!FP8) wait_loads<0>();
        } else {
            auto buf = [&](int t) { return (t & 1) * 2 * TILE * ROW; };
            auto fill = [&](int t) {
                load(false, buf(t) + first_row * ROW);
                load(true, buf(t) + (TILE + first_row) * ROW);
            };
            auto arrive = [&](int t) {
                if constexpr (FP8) {
                    widen(false, buf(t) + first_row * ROW);
                    widen(true, buf(t) + (TILE + first_row) * ROW);
                } else {
                    wait_loads<0>();
                }
                meet();
            };
            bool missing = false, missing_next = false;
            if (tiles > 0) {
                missing = find(0);
                fill(0);
                missing_next = find(min(1, tiles - 1));
                arrive(0);
            }
            // Each wave meets the others once a tile, whichever of the two loops it is in.
            auto step = [&](int t, auto all) {
                const int first = from + t * X::STEP;
                const uint8_t *kb = own + buf(t), *vb = kb + TILE * ROW;
                const bool some = decltype(all)::value || first < most;
                uint32_t there[SUBS];
                if constexpr (!decltype(all)::value)
                    if (some) present(first, missing, there);
                // 8-bit values take registers that the scores' operands need
                if (!FP8 && t + 1 < tiles) fill(t + 1);
                if (some) scores(kb);
                if (FP8 && t + 1 < tiles) fill(t + 1);
                if constexpr (decltype(all)::value) {
                    add(vb, raise(first, all, there));
                } else if (some) {
                    add_with_care(vb, first, there, raise(first, all, there));
                }
                if (t + 1 < tiles) {
                    missing = missing_next;
                    missing_next = find(min(t + 2, tiles - 1));
                    arrive(t + 1);
                }
            };
            int t = 0;
            for (; t < tiles && from + t * X::STEP + TILE <= least && !missing; ++t) step(t, std::true_type());
            for (; t < tiles; ++t) step(t, std::false_type());
        }

        // The piece's result.  One that has all that its lines see is the result; others wait for the join.
        sum += __shfl_xor(sum, 32);
        const bool sole = which && sg.start == 0 && c1 - c0 == units_of(sg);
        const float v_by = FP8 ? c.v_scale[head] : 1.f;
        const uint32_t part0 = begins ? pl.wgs * X::LINES + side.parts[seg] + (head * sg.ranges + range) * sg.tokens * pl.group +
                                            block * X::LINES
                                      : share * X::LINES;
        auto store = [&](int ln, int d, f32x4_sh x, float mm, float total) {  // dims d..d+3 of a line of the block
            const int sl = block * X::LINES + ln;
            const int64_t t = sg.token + sl / pl.group, qh = head * pl.group + sl % pl.group;
            if (sole) {
                x *= total == 0.f ? 0.f : 1.f / total;
                if (total == 0.f) x = f32x4_sh{0.f, 0.f, 0.f, 0.f};  // nothing to attend to, whatever the values are
                if (FP8) x *= v_by;  // by itself: a large factor over the small sum could run over
                *reinterpret_cast<u32x2_kv *>(a.out + t * a.out_ld + qh * DIM + d) =
                    u32x2_kv{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])};
            } else {
                const int64_t at = part0 + ln;
                *reinterpret_cast<f32x4_sh *>(side.o + at * DIM + d) = x;
                if (d == 0) {
                    side.ml[2 * at] = mm;
                    side.ml[2 * at + 1] = total;
                }
            }
        };
        if constexpr (!FEW) {
            if (valid)
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        store(line, 32 * d + 2 * i + 4 * half, f32x4_sh{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]}, m, sum);
        } else {
            float *mine = reinterpret_cast<float *>(own) + col * (DIM + 4) + 4 * half;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<f32x4_sh *>(mine + 32 * d + 2 * i) = f32x4_sh{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
            if (half == 0) {
                lds.m[wave][col] = m;
                lds.l[wave][col] = sum;
            }
            meet();
            for (int i = tid; i < nlines * (DIM / 4); i += SHARED_THREADS) {
                const int ln = i / (DIM / 4), d = i % (DIM / 4) * 4;
                float top = NEG_INF, total = 0.f;
                f32x4_sh x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < SHARED_WAVES; ++w) top = fmaxf(top, lds.m[w][ln]);
#pragma unroll
                for (int w = 0; w < SHARED_WAVES; ++w) {
                    const float mw = lds.m[w][ln], f = mw == top ? 1.f : __builtin_amdgcn_exp2f(mw - top);
                    total += lds.l[w][ln] * f;
                    x += *reinterpret_cast<const f32x4_sh *>(reinterpret_cast<const float *>(lds.pool + w * X::OWN) + ln * (DIM + 4) + d) * f;
                }
                store(ln, d, x, top, total);
            }
        }
        if (u >= u1) return;
        meet();  // the pool and the sums are free
        next_segment();
    }
}

template <int DIM, bool FP8>
__global__ __launch_bounds__(SHARED_THREADS, DIM > 128 ? 1 : 2) void kv_shared_kernel(KvCache c, KvAttendShared a, SharedPlan pl) {
    __shared__ __align__(16) uint8_t pool[std::max(Shape<DIM, FP8, true>::BYTES, Shape<DIM, FP8, false>::BYTES)];
    __shared__ float s_m[SHARED_WAVES][32], s_l[SHARED_WAVES][32];
    const SharedLds lds = {pool, s_m, s_l};
    const SharedPlan::Division dv = *pl.division;
    const int n0 = dv.shares[0], n1 = dv.shares[1], b = (int)blockIdx.x;
    if (b >= n0 + n1) return;
    const int which = b >= n0;
    // Workgroups go to the 8 XCDs in turn; neighbouring shares, which meet the same keys, go to one.
    int share = b - n0;
    if (!which) share = b % 8 * (n0 / 8) + min(b % 8, n0 % 8) + b / 8;
    if (pl.side[which].lines == Shape<DIM, FP8, true>::LINES) attend_share<DIM, FP8, true>(c, a, pl, which, share, which ? n1 : n0, (which ? dv.whole[1] : dv.whole[0]), lds);
    else attend_share<DIM, FP8, false>(c, a, pl, which, share, which ? n1 : n0, (which ? dv.whole[1] : dv.whole[0]), lds);
}

// The last launch: each line's parts, in a fixed order, by a wave.
constexpr int JOIN_THREADS = 256, JOIN_WAVES = 20;  // of a workgroup, and of a CU (24: registers in scratch)
constexpr float PART_BY = 1.f / (1 << 20);  // each part's weights sum to 1 at the most, and there are fewer than 2^20 of them
template <int DIM>
__global__ __launch_bounds__(JOIN_THREADS, JOIN_WAVES / 4) void kv_shared_join_kernel(KvCache c, KvAttendShared a, SharedPlan pl, int each) {
    constexpr int LANES = DIM / 4, SLICES = 64 / LANES;  // lanes of a part, four dims each, and parts taken side by side
    const int lane = threadIdx.x & 63, d = lane % LANES * 4;
    const int wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * (JOIN_THREADS / 64) + (threadIdx.x >> 6)));
    const int all_lines = a.tokens * a.q_heads, last = (int)min((int64_t)(wave + 1) * each, (int64_t)all_lines);
    // Where a run's parts are, 32 ranges of each side at a time, side 0 in lanes 0..31: of each range the part that
    // begins it and those that workgroups begin within it, 3 at the most, a share being more than half of a piece.
    constexpr int RANGES = 32, MOST_PARTS = 4;
    __shared__ uint32_t s_place[JOIN_THREADS / 64][2 * RANGES * MOST_PARTS];
    uint32_t *const places = s_place[threadIdx.x >> 6];
    const int which = lane / RANGES;
    const auto &side = which ? pl.side[1] : pl.side[0];
    const uint32_t wgs_places = pl.wgs * side.lines;
    const int lines_log2 = __builtin_ctz(side.lines);
    const SharedPlan::Division dv = *pl.division;
    const int shares = which ? dv.shares[1] : dv.shares[0];
    const bool whole = which ? dv.whole[1] : dv.whole[0];
    // A row's lines are counted by head, then token and query head, as its parts are.
    for (int at = (int)min((int64_t)wave * each, (int64_t)all_lines); at < last;) {
        const int2 of = pl.tokens[at / a.q_heads];
        if (of.x < 0) {  // of no row
            at += a.q_heads - at % a.q_heads;
            continue;
        }
        Segment sg = {0, 0, 0, 0, 0, 0, 0, 1};
        uint32_t all_cost = 1, first0 = 0, parts0 = 0;
        const int seg = which ? of.x : of.y;
        if (seg >= 0) {
            sg = side.segment[seg];
            all_cost = side.cost[side.segments];
            first0 = side.cost[seg];
            parts0 = side.parts[seg];
            if (sg.tokens == 0) sg.ranges = 0;
        }
        const int token0 = first_token(a, of.x), per_head = (first_token(a, of.x + 1) - token0) * pl.group;
        const int end = min((token0 * a.q_heads) + per_head * c.heads, last);
        if (per_head <= 0 || end <= at) return;  // runs of tokens that are none
        if (__any(which && whole && sg.start == 0 && sg.ranges == 1)) {  // written already
            at = end;
            continue;
        }
        const int reach = sg.reach;
        while (at < end) {
            // A run of lines of a head, in one block of each side.
            const int head = (at - token0 * a.q_heads) / per_head, line = at - token0 * a.q_heads - head * per_head;
            // (Within the segment, whatever the runs of tokens say.)
            const int in = bounded((token0 - sg.token) * pl.group + line, 0, max(sg.tokens * pl.group - 1, 0));
            const int block = in >> lines_log2, nth = which ? nth_of(block, sg.blocks) : block;
            const int left = sg.ranges ? min((block + 1) * side.lines, sg.tokens * pl.group) - in : INT32_MAX;  // of the block
            const int run = min(min(min(__builtin_amdgcn_readlane(left, 0), __builtin_amdgcn_readlane(left, RANGES)), per_head - line),
                                end - at);
            const uint32_t first = first0 + head * head_cost(sg);
            const uint32_t place0 = parts0 + wgs_places + head * sg.ranges * sg.tokens * pl.group + in;
            const int most = max(__builtin_amdgcn_readlane(sg.ranges, 0), __builtin_amdgcn_readlane(sg.ranges, RANGES));
            at += run;
            int parts = 0;
            auto find = [&](int r0) {  // true: written already
                const int r = r0 + lane % RANGES, len = min(reach, units_of(sg) - r * reach);
                int n = 0, w0 = 0;
                if (r < sg.ranges) {
                    n = 1;
                    if (!whole) {  // the shares that its first and its last unit are in
                        const uint32_t u = first + r * sg.blocks * (reach + START) + nth * (len + START) + START;
                        w0 = (int)share_of(u + 1, shares, all_cost, 1.0);
                        n = min((int)share_of(u + len, shares, all_cost, 1.0) - w0 + 1, MOST_PARTS);
                    }
                }
                const int upto = wave_running_sum(n);
                parts = __builtin_amdgcn_readlane(upto, 63);
                if (__any(which && sg.start == 0 && sg.ranges == 1 && n == 1)) return true;
                for (int i = 0; i < n; ++i)
                    places[upto - n + i] = (uint32_t)which << 31 | (i == 0 ? place0 + r * sg.tokens * pl.group
                                                                           : min(w0 + i, shares - 1) * side.lines + (in & (side.lines - 1)));
                __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                __builtin_amdgcn_wave_barrier();
                __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
                return false;
            };
            if (find(0)) continue;
            for (int i = 0; i < run; ++i) {
                float top = NEG_INF, total = 0.f;
                f32x4_sh x = {0.f, 0.f, 0.f, 0.f};
                for (int r0 = 0;;) {
                    constexpr int AHEAD = 4;
                    for (int i0 = 0; i0 < parts; i0 += AHEAD * SLICES) {
                        f32x4_sh y[AHEAD];
                        float2 ml[AHEAD];
#pragma unroll
                        for (int k = 0; k < AHEAD; ++k) {
                            const uint32_t from = places[min(i0 + k * SLICES + lane / LANES, parts - 1)];
                            const auto &f = from >> 31 ? pl.side[1] : pl.side[0];
                            const int64_t place = (from & 0x7FFFFFFFu) + i;
                            ml[k] = *reinterpret_cast<const float2 *>(f.ml + 2 * place);
                            y[k] = *reinterpret_cast<const f32x4_sh *>(f.o + place * DIM + d);
                        }
                        float up = top;
#pragma unroll
                        for (int k = 0; k < AHEAD; ++k) up = fmaxf(up, ml[k].x);
                        const float fade = top == up ? 1.f : __builtin_amdgcn_exp2f(top - up);
                        total *= fade;
                        x *= fade;
                        top = up;
#pragma unroll
                        for (int k = 0; k < AHEAD; ++k)
                            if (i0 + k * SLICES + lane / LANES < parts) {
                                const float f = ml[k].x == top ? 1.f : __builtin_amdgcn_exp2f(ml[k].x - top);
                                total += ml[k].y * f;
                                x += y[k] * (f * PART_BY);
                            }
                    }
                    if (most <= RANGES) break;
                    r0 = r0 + RANGES < most ? r0 + RANGES : 0;
                    __builtin_amdgcn_wave_barrier();
                    find(r0);  // the next ranges, or the first ones for the next line
                    if (r0 == 0) break;
                }
#pragma unroll
                for (int s = LANES; s < 64; s <<= 1) {
                    const float other = __shfl_xor(top, s), up = fmaxf(top, other);
                    const float f = top == up ? 1.f : __builtin_amdgcn_exp2f(top - up);
                    const float g = other == up ? 1.f : __builtin_amdgcn_exp2f(other - up);
                    total = total * f + __shfl_xor(total, s) * g;
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[e] = x[e] * f + __shfl_xor(x[e], s) * g;
                    top = up;
                }
                x *= total == 0.f ? 0.f : 1.f / (total * PART_BY);
                if (total == 0.f) x = f32x4_sh{0.f, 0.f, 0.f, 0.f};  // nothing to attend to, whatever the values are
                if (c.fp8) x *= c.v_scale[head];
                const int64_t token = token0 + (line + i) / pl.group, qh = head * pl.group + (line + i) % pl.group;
                if (lane < LANES)
                    *reinterpret_cast<u32x2_kv *>(a.out + token * a.out_ld + qh * DIM + d) =
                        u32x2_kv{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])};
            }
        }
    }
}

// The plan, its scratch laid out from `base`; returns the bytes (-1: more than a launch takes).
static int64_t shared_plan(const KvCache &c, int q_heads, int tokens, int groups, int max_len, bool all_bits, int cu_count,
                           uint8_t *base, SharedPlan *pl) {
    if ((((int64_t)c.pages * c.heads) << c.page_log2) * (c.dim / 8) >> 32) return -1;  // a pool's pieces are counted in 32 bits
    pl->group = q_heads / c.heads;
    const int64_t lines = (int64_t)tokens * pl->group, chunks = (max_len + UNIT - 1) / UNIT;
    int64_t units = 0;
    for (int which = 0; which < 2; ++which) {
        auto &side = pl->side[which];
        side.segments = which ? c.rows : groups;
        // Few lines cost least where a block has them all, and half again as much with one line more; many, in blocks of 128, cost about
        // the same up to 128.  Calls with blocks of 32 and 128 lines: 16 rows of 8192 slots, 32 lines each 116 and 123 us (8 bits 70 and
        // 103), 36 lines 171 and 124 (106 and 103), 128 lines 339 and 143; 16 rows of 4096 of 256 dims, 32 lines 121 and 136, 36 lines 173 and 136; a
        // prefix of 16384, 32 lines 43 and 42, 64 lines 44 and 46, 256 lines 76 and 69.  The mean decides, as the lines of each segment are on the
        // device: 63 single tokens over 4096 slots beside a prompt's 512 over 2048 (mean 36) 240 and 246, 15 over 8192 beside
        // 2048 over 4096 (516) 510 and 267, 500 over 2048 beside 300 (6) 737 and 865.
        const int64_t mean = side.segments ? (lines + side.segments - 1) / side.segments : 0;  // lines of a segment
        side.lines = mean <= 32 || all_bits ? 32 : 128;
        if (side.segments) units += (lines / side.lines + side.segments) * c.heads * chunks;
        if (units > INT32_MAX / (1 + START)) return -1;
    }
    // As many workgroups as run at once: two on a CU, one at 256 dims (registers, LDS).
    pl->wgs = (int)std::min<int64_t>(units, (int64_t)cu_count * (c.dim > 128 ? 1 : 2));
    if (!fits_launch(((int64_t)tokens * q_heads + 3) / 4, JOIN_THREADS)) return -1;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        uint8_t *p = base ? base + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    pl->tokens = (int2 *)take((int64_t)tokens * 8);
    pl->sees = (int32_t *)take((int64_t)tokens * 4);
    pl->division = (SharedPlan::Division *)take(sizeof(SharedPlan::Division));
    for (int which = 0; which < 2; ++which) {
        auto &side = pl->side[which];
        side.segment = (Segment *)take((int64_t)side.segments * sizeof(Segment));
        side.cost = (uint32_t *)take(((int64_t)side.segments + 1) * 4);
        side.parts = (uint32_t *)take((int64_t)side.segments * 4);
        // A line for each that a workgroup may begin within a piece; and by segment, head, range and line: with
        // ranges no longer than needed, a block more for each workgroup than the lines there are.
        side.places = side.segments ? 2u * pl->wgs * side.lines + (uint32_t)tokens * q_heads : 0;
        side.ml = (float *)take((int64_t)side.places * 8);
        side.o = (float *)take((int64_t)side.places * c.dim * 4);
    }
    return at;
}

int64_t kv_attend_shared_workspace_bytes(const KvCache &c, int q_heads, int tokens, int groups, int max_len, bool all_bits,
                                         int cu_count) {
    SharedPlan pl;
    return shared_plan(c, q_heads, tokens, groups, max_len, all_bits, cu_count, nullptr, &pl);
}

template <int DIM>
static void launch_shared(const KvCache &c, const KvAttendShared &a, const SharedPlan &pl, int cu_count, hipStream_t stream) {
    const dim3 grid((unsigned)pl.wgs), threads(SHARED_THREADS);
    if (c.fp8) hipLaunchKernelGGL((kv_shared_kernel<DIM, true>), grid, threads, 0, stream, c, a, pl);
    else hipLaunchKernelGGL((kv_shared_kernel<DIM, false>), grid, threads, 0, stream, c, a, pl);
    // A wave for each line, up to as many as run at once; then each wave takes several, of few tokens.
    const int64_t lines = (int64_t)a.tokens * a.q_heads, most = (int64_t)cu_count * JOIN_WAVES;
    const int each = (int)((lines + most - 1) / most);
    const unsigned wgs = (unsigned)((lines + (int64_t)each * (JOIN_THREADS / 64) - 1) / ((int64_t)each * (JOIN_THREADS / 64)));
    hipLaunchKernelGGL((kv_shared_join_kernel<DIM>), dim3(wgs), dim3(JOIN_THREADS), 0, stream, c, a, pl, each);
}

hipError_t launch_kv_attend_shared(const KvCache &c, const KvAttendShared &a, int cu_count, hipStream_t stream) {
    SharedPlan pl;
    shared_plan(c, a.q_heads, a.tokens, a.groups, a.max_len, a.all_bits, cu_count, a.ws, &pl);
    const unsigned finders = (unsigned)((a.tokens + PLAN_THREADS - 1) / PLAN_THREADS);
    hipLaunchKernelGGL(kv_shared_plan_kernel, dim3(finders + 1), dim3(PLAN_THREADS), 0, stream, c, a, pl);
    switch (c.dim) {
    case 64: launch_shared<64>(c, a, pl, cu_count, stream); break;
    case 128: launch_shared<128>(c, a, pl, cu_count, stream); break;
    default: launch_shared<256>(c, a, pl, cu_count, stream); break;
    }
    return hipGetLastError();
}

}  // namespace nbw
