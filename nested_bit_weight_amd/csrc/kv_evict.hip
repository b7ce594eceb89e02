// kv_evict.hip -- eviction from the cache by accumulated attention weight,
// gfx950.
//
// For each (row, head) of n > budget slots: the budget largest keys stay, the
// lowest slot first among equals, and the kept rows past the budget move into
// the places below it that became free.  Ranking reads 8 bytes a slot and
// moves copy 4 * dim elements a moved row, so the two are separate problems:
//
//  - Ranking.  Up to 16384 slots one workgroup takes a (row, head), with its keys
//    in registers, up to 16 a thread.  The budget-th largest key is found by counting: a
//    histogram of 2048 bins over the 11 bits below the leading bits that all
//    candidates share, the bin that holds the wanted key, and again inside it,
//    until a bin is wanted whole or holds one value.  On attention totals the first
//    two passes do.  Protected slots, which all share the largest key, are only
//    counted.  (Bins over fixed leading bits put most totals, alike in sign and
//    exponent, into a few bins, whose atomics then wait for each other.)
//    A slot's place in the list of gaps (below the budget, not kept) or movers
//    (past it, kept) is the number of them in lower slots: ballots within a
//    wave, and one running sum over the waves' counts.
//  - Longer rows are more than one CU reads in good time (one row of 120001 slots
//    in 8 workgroups: 160 us).  There a workgroup takes 4096 slots of a (row, head)
//    and the steps above are launches of their own: newest position, keys and a
//    histogram over their upper 11 bits, two more over the next 11 and the last 10
//    of those in the wanted bin, counts, lists.  Histograms meet in integer
//    atomics, whose order does not matter.
//  - Moves need the whole device: with more than a few a last launch makes them, 16
//    to a workgroup.  In the steady state of one token over the budget the ranking's
//    workgroup makes its one move itself.
//
// A move reads at or past the budget and writes below it, so moves never meet,
// and no buffer that the ranking reads is written.
//
// Measured (8 heads of 128): 32 rows one over a budget of 2048: 7.0 us, latency;
// 12 rows of up to 16384 brought down to 4096 (247 MB): 72 us, 20 of them the ranking
// on 96 CUs and 52 the moves, 4.4 TB/s in rows of 256 bytes (a plain copy: 4.9); one
// row of 120001 in 8 bits brought down to 16384: 49 us, 18 of them the moves and the
// rest six launches, each a few dependent loads long.
#include <algorithm>

#include "kv.h"

namespace nbw {

typedef float f32x4_ev __attribute__((ext_vector_type(4)));
typedef int32_t i32x4_ev __attribute__((ext_vector_type(4)));

constexpr int EVICT_BINS_LOG2 = 11, EVICT_BINS = 1 << EVICT_BINS_LOG2;
constexpr uint32_t KEY_HELD = 0xFFFFFFFFu, KEY_NEG_INF = 0x007FFFFFu;  // protected: above +infinity's, 0xFF800000
constexpr int EVICT_ROW = 16384;     // the longest row that one workgroup ranks (32 keys a thread spill: at 32768 both ways took 46-49 us)
constexpr int PART_THREADS = 256, PART_GROUPS = 4, PART = PART_THREADS * PART_GROUPS * 4;  // longer ones: slots of a workgroup
constexpr int MOVES = 16;           // moves of a workgroup of the second launch
constexpr int FUSED_MOVES = 64;     // up to so many the ranking's workgroup makes itself
constexpr int FEW_OUT = 4;          // up to so many slots over the budget are found one by one

// The workspace: the lists of each (row, head) and their lengths; for long rows,
// what the launches leave each other.
struct EvictPlan {
    int32_t *lists;   // [rows * heads][2][most]: places to move to, slots to move from
    int most;
    int32_t *counts;  // [rows * heads]; both null where the ranking's workgroup moves
    int vec;          // totals and positions may be read 16 bytes at a time
    int parts;        // parts of a long row; 0: one workgroup ranks
    uint32_t *keys;   // [rows * heads][parts * PART]
    int32_t *newest;  // [rows * heads][parts]
    int32_t *hist;    // [rows * heads][3][EVICT_BINS]
    int32_t *found;   // [rows * heads][3][3]: each histogram's bin, keys above it, keys in it
    int32_t *tally;   // [rows * heads][parts][4]: keys above the limit and equal to it, below the budget and past it
};

// Keys as unsigned numbers of the same order.  -0 and +0 are equal.
__device__ __forceinline__ uint32_t evict_key(float acc, int32_t pos, int32_t newest, const KvEvict &a) {
    if (pos < a.sink || (int64_t)pos > (int64_t)newest - a.recent) return KEY_HELD;
    if (acc != acc) return KEY_NEG_INF;
    const uint32_t u = __float_as_uint(acc == 0.f ? 0.f : acc);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// `count` moves of one (row, head): the 16-byte pieces of each move's key and
// value, and its total and position.
template <int ROW_BYTES, int THREADS, bool NT>
__device__ __forceinline__ void make_moves(const KvCache &c, const KvEvict &a, int row, int head, const int32_t *to,
                                           const int32_t *of, int count) {
    constexpr int VECS = ROW_BYTES / 16, AT_ONCE = 2;
    const int64_t base = ((int64_t)row * c.heads + head) * c.cap;
    const int end = count * VECS;  // at most MOVES or FUSED_MOVES rows
    for (int i0 = threadIdx.x; i0 < end; i0 += THREADS * AT_ONCE) {
        int64_t src[AT_ONCE], dst[AT_ONCE];
        u32x4_kv k[AT_ONCE], v[AT_ONCE];
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j) {
            const int i = i0 + j * THREADS;
            src[j] = dst[j] = -1;
            if (i < end) {
                const int m = i / VECS, t = to[m], f = of[m];
                src[j] = kv_row(c, row, head, f);
                dst[j] = kv_row(c, row, head, t);
                if (i % VECS == 0) {
                    a.acc_out[base + t] = a.acc[base + f];
                    a.pos_out[base + t] = a.pos[base + f];
                }
            }
        }
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j)
            if (src[j] >= 0 && dst[j] >= 0) {
                const int64_t at = src[j] * ROW_BYTES + (i0 + j * THREADS) % VECS * 16;
                const u32x4_kv *kp = reinterpret_cast<const u32x4_kv *>(c.k + at), *vp = reinterpret_cast<const u32x4_kv *>(c.v + at);
                k[j] = NT ? __builtin_nontemporal_load(kp) : *kp;
                v[j] = NT ? __builtin_nontemporal_load(vp) : *vp;
            }
#pragma unroll
        for (int j = 0; j < AT_ONCE; ++j)
            if (src[j] >= 0 && dst[j] >= 0) {
                const int64_t at = dst[j] * ROW_BYTES + (i0 + j * THREADS) % VECS * 16;
                *reinterpret_cast<u32x4_kv *>(c.k + at) = k[j];
                *reinterpret_cast<u32x4_kv *>(c.v + at) = v[j];
            }
    }
}

// Four values from j on (j a multiple of 4), those from `end` on as `none`.
template <class V>
struct Four { V v[4]; };
template <class V>
__device__ __forceinline__ Four<V> four(const V *p, int j, int end, V none, bool vec) {
    typedef V vec_t __attribute__((ext_vector_type(4)));
    Four<V> r = {{none, none, none, none}};
    if (vec && j + 4 <= end) {
        const vec_t w = *reinterpret_cast<const vec_t *>(p + j);
#pragma unroll
        for (int e = 0; e < 4; ++e) r.v[e] = w[e];
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < end) r.v[e] = p[j + e];
    }
    return r;
}

// Totals x and positions y of slots j .. j + 3 below `end`, of the (row, head) at `base`, to the outputs.
__device__ __forceinline__ void put_out(const KvEvict &a, int64_t base, int j, int end, const Four<float> &x,
                                        const Four<int32_t> &y, bool vec) {
    if (vec && j + 4 <= end) {
        *reinterpret_cast<f32x4_ev *>(a.acc_out + base + j) = f32x4_ev{x.v[0], x.v[1], x.v[2], x.v[3]};
        *reinterpret_cast<i32x4_ev *>(a.pos_out + base + j) = i32x4_ev{y.v[0], y.v[1], y.v[2], y.v[3]};
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (j + e < end) {
                a.acc_out[base + j + e] = x.v[e];
                a.pos_out[base + j + e] = y.v[e];
            }
    }
}
__device__ __forceinline__ void copy_out(const KvEvict &a, int64_t base, int j, int end, bool vec) {
    if (j < end) put_out(a, base, j, end, four(a.acc + base, j, end, 0.f, vec), four(a.pos + base, j, end, 0, vec), vec);
}

// The bin of `hist` that the want-th largest key is in: found = {bin, keys above
// it, keys in it}.  Every thread gets the same answer.
template <int THREADS>
__device__ __forceinline__ void find_bin(const int *hist, int want, int *red, int *found) {
    constexpr int WAVES = THREADS / 64, PER = EVICT_BINS / THREADS;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // Bins from the top: this thread's are PER of them below tid * PER others.
    int count[PER], mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        count[i] = hist[EVICT_BINS - 1 - (tid * PER + i)];
        mine += count[i];
    }
    int upto = wave_running_sum(mine);
    if (lane == 63) red[wave] = upto;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WAVES; ++w)
        if (w < wave) upto += red[w];
    int above = upto - mine;
    if (above < want && want <= upto) {
        bool open = true;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (open && want <= above + count[i]) {
                found[0] = EVICT_BINS - 1 - (tid * PER + i);
                found[1] = above;
                found[2] = count[i];
                open = false;
            }
            above += count[i];
        }
    }
    __syncthreads();
}

// What stays: the keys above `limit`, and of its equals the first `want` in the
// order of the slots; with `all`, every one.
struct Limit {
    uint32_t key;
    int want;
    bool all;
};

// The lists' entries of one workgroup's keys, slots first .. first + THREADS *
// GROUPS * 4 - 1 (thread t has four from first + 4 (g THREADS + t) on).  equals,
// gaps, movers: how many there are in lower slots; returns the movers up to and
// with these.
template <int THREADS, int GROUPS>
__device__ __forceinline__ int list_moves(const uint32_t (&key)[GROUPS][4], int b, int first, const Limit &lim, int equals,
                                          int gaps, int movers, int32_t *to, int32_t *of) {
    constexpr int WAVES = THREADS / 64, TAB = GROUPS * WAVES;  // the waves' counts in the order of the slots
    __shared__ int tab[2][TAB + 1];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint64_t lower = (1ull << lane) - 1;
    // The running sums over `tab`: entry i becomes the sum of those before it, the last one the total.
    auto sums = [&]() {
        __syncthreads();
        if (wave < 2) {
            int carry = 0;
#pragma unroll
            for (int i0 = 0; i0 < TAB; i0 += 64) {
                const int i = i0 + lane, x = i < TAB ? tab[wave][i] : 0;
                const int s = wave_running_sum(x);
                if (i < TAB) tab[wave][i] = carry + s - x;
                carry += __builtin_amdgcn_readlane(s, 63);
            }
            if (lane == 0) tab[wave][TAB] = carry;
        }
        __syncthreads();
    };
    uint32_t keep = 0;  // bit 4 g + e
#pragma unroll
    for (int g = 0; g < GROUPS; ++g)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            keep |= (uint32_t)(key[g][e] > lim.key || (lim.all && key[g][e] == lim.key)) << (4 * g + e);
    if (!lim.all) {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            int count = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) count += __popcll(__ballot(key[g][e] == lim.key));
            if (lane == 0) tab[0][g * WAVES + wave] = tab[1][g * WAVES + wave] = count;
        }
        sums();
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            int r = equals + tab[0][g * WAVES + wave];
#pragma unroll
            for (int e = 0; e < 4; ++e) r += __popcll(__ballot(key[g][e] == lim.key) & lower);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (key[g][e] == lim.key) keep |= (uint32_t)(r++ < lim.want) << (4 * g + e);
        }
        __syncthreads();
    }
    auto slot_of = [&](int g) { return first + (g * THREADS + tid) * 4; };
    auto is_gap = [&](int g, int e) { return !(keep >> (4 * g + e) & 1) && slot_of(g) + e < b; };
    auto is_mover = [&](int g, int e) { return (keep >> (4 * g + e) & 1) && slot_of(g) + e >= b; };
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        int count_g = 0, count_m = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            count_g += __popcll(__ballot(is_gap(g, e)));
            count_m += __popcll(__ballot(is_mover(g, e)));
        }
        if (lane == 0) {
            tab[0][g * WAVES + wave] = count_g;
            tab[1][g * WAVES + wave] = count_m;
        }
    }
    sums();
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
        int rg = gaps + tab[0][g * WAVES + wave], rm = movers + tab[1][g * WAVES + wave];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            rg += __popcll(__ballot(is_gap(g, e)) & lower);
            rm += __popcll(__ballot(is_mover(g, e)) & lower);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (is_gap(g, e)) to[rg++] = slot_of(g) + e;
            if (is_mover(g, e)) of[rm++] = slot_of(g) + e;
        }
    }
    return movers + tab[1][TAB];
}

// Rows of up to THREADS * GROUPS * 4 slots: one workgroup for each (row, head).
template <int THREADS, int GROUPS>
__global__ __launch_bounds__(THREADS) void kv_evict_kernel(KvCache c, KvEvict a, EvictPlan pl) {
    constexpr int WAVES = THREADS / 64;
    __shared__ int hist[EVICT_BINS];
    __shared__ int red[3][WAVES];
    __shared__ int found[3];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int row = blockIdx.x / c.heads, head = blockIdx.x % c.heads;
    const int n = kv_len(a.lens, row, a.max_len), b = a.budget;
    const int64_t base = (int64_t)blockIdx.x * c.cap;
    if (head == 0 && tid == 0) a.lens_out[row] = n < b ? n : b;
    if (n <= b) {
        if (pl.counts && tid == 0) pl.counts[blockIdx.x] = 0;
        for (int j = tid * 4; j < n; j += THREADS * 4) copy_out(a, base, j, n, pl.vec);
        return;
    }

    // The newest position, then the keys; how many are protected and the range of the rest.
    uint32_t key[GROUPS][4];
    auto slot_of = [&](int g) { return (g * THREADS + tid) * 4; };
    int32_t newest = INT32_MIN;
    int held = 0;
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    {
        Four<float> x[GROUPS];
        Four<int32_t> y[GROUPS];
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) y[g] = four(a.pos + base, slot_of(g), n, INT32_MIN, pl.vec);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) x[g] = four(a.acc + base, slot_of(g), n, 0.f, pl.vec);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) newest = max(newest, y[g].v[e]);
        newest = wave_max(newest);
        if (lane == 0) red[0][wave] = newest;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) newest = max(newest, red[0][w]);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)  // what goes is overwritten when its place is taken
            if (slot_of(g) < b) put_out(a, base, slot_of(g), b, x[g], y[g], pl.vec);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool there = slot_of(g) + e < n;
                const uint32_t k = there ? evict_key(x[g].v[e], y[g].v[e], newest, a) : 0;  // 0: below every key
                key[g][e] = k;
                held += k == KEY_HELD;
                if (there && k != KEY_HELD) {
                    lo = min(lo, k);
                    hi = max(hi, k);
                }
            }
    }
    __shared__ int32_t few[2][FUSED_MOVES];
    int32_t *to = pl.counts ? pl.lists + (int64_t)blockIdx.x * 2 * pl.most : few[0], *of = pl.counts ? to + pl.most : few[1];
    int movers;
    if (n - b <= FEW_OUT) {
        // The few that go, one after the other: the smallest key, among equals the
        // highest slot.
        __shared__ uint64_t least[FEW_OUT][WAVES];
        int out[FEW_OUT];
#pragma unroll
        for (int i = 0; i < FEW_OUT; ++i) {
            out[i] = INT32_MAX;
            if (i >= n - b) continue;
            uint32_t low = ~0u, rest = ~0u;  // the key, and how far its slot is from the end
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (key[g][e]) low = min(low, key[g][e]);
            low = wave_min_u(low);
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (key[g][e] == low) rest = (uint32_t)(INT32_MAX - (slot_of(g) + e));  // slots ascend
            uint64_t m = (uint64_t)low << 32 | wave_min_u(rest);
            if (lane == 0) least[i][wave] = m;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WAVES; ++w) m = min(m, least[i][w]);
            out[i] = INT32_MAX - (int)(uint32_t)m;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (slot_of(g) + e == out[i]) key[g][e] = 0;
        }
        movers = 0;  // as many as gaps
#pragma unroll
        for (int i = 0; i < FEW_OUT; ++i) movers += out[i] < b;
        if (tid == 0) {
            int gaps = 0, from = b;
            for (int last = -1; gaps < movers;) {  // the gaps in ascending order, each with the next slot that stays
                int next = INT32_MAX;
#pragma unroll
                for (int i = 0; i < FEW_OUT; ++i)
                    if (out[i] > last) next = min(next, out[i]);
                last = next;
                bool goes;
                do {
                    goes = false;
#pragma unroll
                    for (int i = 0; i < FEW_OUT; ++i) goes |= out[i] == from;
                    from += goes;
                } while (goes);
                to[gaps] = next;
                of[gaps++] = from++;
            }
        }
    } else {
        __syncthreads();
        held = wave_sum(held);
        lo = wave_min_u(lo);
        hi = wave_max_u(hi);
        if (lane == 0) {
            red[0][wave] = held;
            red[1][wave] = (int)lo;
            red[2][wave] = (int)hi;
        }
        __syncthreads();
        held = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            held += red[0][w];
            lo = min(lo, (uint32_t)red[1][w]);
            hi = max(hi, (uint32_t)red[2][w]);
        }

        Limit lim = {KEY_HELD, b, held == b};
        if (held < b) {
            lim.want = b - held;
            while (lo != hi) {  // the want-th largest of the keys within [lo, hi]
                const int bits = 32 - __builtin_clz(lo ^ hi);
                const int shift = bits > EVICT_BINS_LOG2 ? bits - EVICT_BINS_LOG2 : 0;
                for (int i = tid; i < EVICT_BINS; i += THREADS) hist[i] = 0;
                __syncthreads();
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t k = key[g][e];
                        if (k >= lo && k <= hi) atomicAdd(&hist[(k >> shift) & (EVICT_BINS - 1)], 1);
                    }
                __syncthreads();
                find_bin<THREADS>(hist, lim.want, red[0], found);
                const uint32_t low = (((hi >> shift) & ~(uint32_t)(EVICT_BINS - 1)) | (uint32_t)found[0]) << shift;
                const uint32_t high = low + ((1u << shift) - 1);
                lim.want -= found[1];
                lim.all = found[2] == lim.want;
                lo = max(lo, low);
                hi = min(hi, high);
                if (lim.all || shift == 0) break;
                __syncthreads();  // found and hist are free
            }
            lim.key = lo;
        }

        movers = list_moves<THREADS, GROUPS>(key, b, 0, lim, 0, 0, 0, to, of);
    }
    if (pl.counts) {
        if (tid == 0) pl.counts[blockIdx.x] = movers;
        return;
    }
    __syncthreads();  // the lists are written
    switch (c.fp8 ? c.dim : 2 * c.dim) {
    case 64: make_moves<64, THREADS, false>(c, a, row, head, to, of, movers); break;
    case 128: make_moves<128, THREADS, false>(c, a, row, head, to, of, movers); break;
    case 256: make_moves<256, THREADS, false>(c, a, row, head, to, of, movers); break;
    default: make_moves<512, THREADS, false>(c, a, row, head, to, of, movers); break;
    }
}

// The bits of a key that histogram `level` of a long row counts, and those above them.
__device__ __forceinline__ int level_shift(int level) { return level == 0 ? 21 : level == 1 ? 10 : 0; }

// A long row's limit after `levels` histograms: found[level] holds each one's bin,
// the keys above it and the keys in it.  The prefix of the keys still wanted and how
// many of them; all: they are wanted whole (later histograms are then not made).
__device__ __forceinline__ Limit limit_after(const int32_t *found, int levels, int budget) {
    Limit lim = {0, budget, false};
    for (int l = 0; l < levels && !lim.all; ++l) {
        lim.key |= (uint32_t)found[3 * l] << level_shift(l);
        lim.want -= found[3 * l + 1];
        lim.all = found[3 * l + 2] == lim.want;
    }
    return lim;
}

enum EvictStage { NEWEST, COUNT0, COUNT1, COUNT2, TALLY, LIST };

// One step of a long row's ranking: workgroup = (row, head, part of PART slots).
template <int STAGE>
__global__ __launch_bounds__(PART_THREADS) void kv_evict_part_kernel(KvCache c, KvEvict a, EvictPlan pl) {
    constexpr int THREADS = PART_THREADS, GROUPS = PART_GROUPS, WAVES = THREADS / 64;
    __shared__ int hist[EVICT_BINS];
    __shared__ int red[4][WAVES];
    __shared__ int found[3];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int which = blockIdx.x / pl.parts, part = blockIdx.x % pl.parts, first = part * PART;
    const int row = which / c.heads, head = which % c.heads;
    const int n = kv_len(a.lens, row, a.max_len), b = a.budget;
    const int64_t base = (int64_t)which * c.cap;
    int32_t *ghist = pl.hist + (int64_t)which * 3 * EVICT_BINS, *gfound = pl.found + (int64_t)which * 9;
    auto slot_of = [&](int g) { return first + (g * THREADS + tid) * 4; };
    if (STAGE == LIST && part == 0 && tid == 0) {
        if (head == 0) a.lens_out[row] = n < b ? n : b;
        if (n <= b && pl.counts) pl.counts[which] = 0;
    }
    if (n <= b) {
        if (STAGE == LIST)
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) copy_out(a, base, slot_of(g), n, pl.vec);
        return;
    }
    if (STAGE == NEWEST) {  // and the histograms' first zeros
        for (int i = part * THREADS + tid; i < 3 * EVICT_BINS; i += pl.parts * THREADS) ghist[i] = 0;
    }
    if (first >= n) {
        if (STAGE == NEWEST && tid == 0) pl.newest[(int64_t)which * pl.parts + part] = INT32_MIN;
        return;
    }
    if (STAGE == NEWEST) {
        int32_t newest = INT32_MIN;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const Four<int32_t> y = four(a.pos + base, slot_of(g), n, INT32_MIN, pl.vec);
#pragma unroll
            for (int e = 0; e < 4; ++e) newest = max(newest, y.v[e]);
        }
        newest = wave_max(newest);
        if (lane == 0) red[0][wave] = newest;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) newest = max(newest, red[0][w]);
        if (tid == 0) pl.newest[(int64_t)which * pl.parts + part] = newest;
        return;
    }

    uint32_t key[GROUPS][4];
    uint32_t *stored = pl.keys + (int64_t)which * pl.parts * PART;
    if (STAGE == COUNT0) {
        Four<float> x[GROUPS];
        Four<int32_t> y[GROUPS];
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) y[g] = four(a.pos + base, slot_of(g), n, INT32_MIN, pl.vec);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) x[g] = four(a.acc + base, slot_of(g), n, 0.f, pl.vec);
        int32_t newest = INT32_MIN;
        for (int i = tid; i < pl.parts; i += THREADS) newest = max(newest, pl.newest[(int64_t)which * pl.parts + i]);
        newest = wave_max(newest);
        if (lane == 0) red[0][wave] = newest;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) newest = max(newest, red[0][w]);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const int j = slot_of(g);
#pragma unroll
            for (int e = 0; e < 4; ++e) key[g][e] = j + e < n ? evict_key(x[g].v[e], y[g].v[e], newest, a) : 0;
            if (j < b) put_out(a, base, j, b, x[g], y[g], pl.vec);  // what goes is overwritten when its place is taken
            *reinterpret_cast<i32x4_ev *>(stored + j) = i32x4_ev{(int)key[g][0], (int)key[g][1], (int)key[g][2], (int)key[g][3]};
        }
    } else {
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const i32x4_ev w = *reinterpret_cast<const i32x4_ev *>(stored + slot_of(g));
#pragma unroll
            for (int e = 0; e < 4; ++e) key[g][e] = (uint32_t)w[e];
        }
    }

    // The last histogram's bin (part 0 leaves it for the launches after this one).
    constexpr int LEVEL = STAGE == COUNT0 ? 0 : STAGE == COUNT1 ? 1 : STAGE == COUNT2 ? 2 : 3;  // histograms made before
    Limit lim = limit_after(gfound, LEVEL - 1, b);
    if (STAGE != COUNT0 && STAGE != LIST && !lim.all) {
        for (int i = tid; i < EVICT_BINS; i += THREADS) hist[i] = ghist[(LEVEL - 1) * EVICT_BINS + i];
        __syncthreads();
        find_bin<THREADS>(hist, lim.want, red[0], found);
        lim.key |= (uint32_t)found[0] << level_shift(LEVEL - 1);
        lim.want -= found[1];
        lim.all = found[2] == lim.want;
        if (part == 0 && tid < 3) gfound[3 * (LEVEL - 1) + tid] = found[tid];
        __syncthreads();
    }
    if (STAGE == LIST) lim = limit_after(gfound, 3, b);

    if (STAGE == COUNT0 || STAGE == COUNT1 || STAGE == COUNT2) {
        if (lim.all) return;
        for (int i = tid; i < EVICT_BINS; i += THREADS) hist[i] = 0;
        __syncthreads();
        int held = 0;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t k = key[g][e];
                if (STAGE == COUNT0) {  // all protected slots' key is counted apart
                    if (k == KEY_HELD) ++held;
                    else if (k) atomicAdd(&hist[k >> 21], 1);
                } else if (k >> level_shift(LEVEL - 1) == lim.key >> level_shift(LEVEL - 1)) {
                    atomicAdd(&hist[(k >> level_shift(LEVEL)) & (STAGE == COUNT1 ? 2047 : 1023)], 1);
                }
            }
        if (STAGE == COUNT0) {
            held = wave_sum(held);
            if (lane == 0 && held) atomicAdd(&hist[KEY_HELD >> 21], held);
        }
        __syncthreads();
        for (int i = tid; i < EVICT_BINS; i += THREADS)
            if (hist[i]) atomicAdd(&ghist[LEVEL * EVICT_BINS + i], hist[i]);
        return;
    }

    if (STAGE == TALLY) {
        int count[4] = {0, 0, 0, 0};
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool past = slot_of(g) + e >= b;
                if (key[g][e] > lim.key) ++count[past];
                else if (key[g][e] == lim.key) ++count[2 + past];
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            count[i] = wave_sum(count[i]);
            if (lane == 0) red[i][wave] = count[i];
        }
        __syncthreads();
        if (tid < 4) {
            int sum = 0;
            for (int w = 0; w < WAVES; ++w) sum += red[tid][w];
            pl.tally[((int64_t)which * pl.parts + part) * 4 + tid] = sum;
        }
        return;
    }

    // LIST: what the parts before this one keep.
    if (wave == 0) {
        int equals = 0, below = 0, past = 0;  // equals, and kept below the budget and past it, in earlier parts
        for (int i0 = 0; i0 < part; i0 += 64) {
            const int i = i0 + lane;
            i32x4_ev t = {0, 0, 0, 0};
            if (i < part) t = *reinterpret_cast<const i32x4_ev *>(pl.tally + ((int64_t)which * pl.parts + i) * 4);
            const int upto = wave_running_sum(t[2] + t[3]);
            const int left = lim.all ? INT32_MAX : max(0, lim.want - (equals + upto - t[2] - t[3]));  // for this part's equals
            const int low = min(t[2], left), high = min(t[3], left - low);
            below += wave_sum(t[0] + low);
            past += wave_sum(t[1] + high);
            equals += __builtin_amdgcn_readlane(upto, 63);
        }
        if (lane == 0) {
            found[0] = equals;
            found[1] = min(first, b) - below;
            found[2] = past;
        }
    }
    __syncthreads();
    int32_t *to = pl.lists + (int64_t)which * 2 * pl.most, *of = to + pl.most;
    const int movers = list_moves<THREADS, GROUPS>(key, b, first, lim, found[0], found[1], found[2], to, of);
    if (first + PART >= n && tid == 0) pl.counts[which] = movers;
}

template <int ROW_BYTES, bool NT>
__global__ __launch_bounds__(256) void kv_move_kernel(KvCache c, KvEvict a, EvictPlan pl, int parts) {
    const int which = blockIdx.x / parts, count = pl.counts[which];
    const int32_t *to = pl.lists + (int64_t)which * 2 * pl.most;
    for (int64_t first = (int64_t)(blockIdx.x % parts) * MOVES; first < count; first += (int64_t)parts * MOVES)
        make_moves<ROW_BYTES, 256, NT>(c, a, which / c.heads, which % c.heads, to + first, to + pl.most + first,
                                       (int)min((int64_t)MOVES, count - first));
}

// Threads of the workgroup that ranks one (row, head): the smallest that holds the longest
// row's keys, 4, 8 or 16 a thread.  The same for every batch: calls in a graph, one token over
// the budget, 256 threads with 16 keys against 512 with 8: 64 (row, head) of 2049 slots 5.8 and
// 5.0 us, 256 of them 6.2 and 5.5, 768 of them 9.0 and 8.7, 512 of 1025 slots 6.4 and 5.9, 768 of
// those 7.0 and 7.2; 768 of 2049 brought down to half 59 both.
static int ranking_threads(int max_len) { return max_len <= 1024 ? 256 : max_len <= 4096 ? 512 : 1024; }

static int64_t evict_plan(const KvCache &c, int budget, int max_len, uint8_t *base, EvictPlan *pl) {  // -1: more than a launch takes
    const int64_t lists = (int64_t)c.rows * c.heads;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        uint8_t *p = base ? base + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    *pl = EvictPlan{};
    pl->most = std::max(0, std::min(budget, max_len - budget));
    if (max_len > EVICT_ROW) pl->parts = (max_len + PART - 1) / PART;
    if (!(pl->parts ? fits_launch(lists * pl->parts, PART_THREADS) : fits_launch(lists, ranking_threads(max_len)))) return -1;
    if (pl->most) {
        if (pl->parts || pl->most > FUSED_MOVES) {
            pl->lists = (int32_t *)take(lists * 2 * pl->most * 4);
            pl->counts = (int32_t *)take(lists * 4);
        }
    }
    if (pl->parts) {
        pl->keys = (uint32_t *)take(lists * pl->parts * PART * 4);
        pl->newest = (int32_t *)take(lists * pl->parts * 4);
        pl->hist = (int32_t *)take(lists * 3 * EVICT_BINS * 4);
        pl->found = (int32_t *)take(lists * 9 * 4);
        pl->tally = (int32_t *)take(lists * pl->parts * 4 * 4);
    }
    return at;
}

int64_t kv_evict_workspace_bytes(const KvCache &c, int budget, int max_len) {
    EvictPlan pl;
    return evict_plan(c, budget, max_len, nullptr, &pl);
}

template <int ROW_BYTES>
static void launch_moves(const KvCache &c, const KvEvict &a, const EvictPlan &pl, hipStream_t stream) {
    // A workgroup for each 16 moves, or for several times 16 where a launch does not take as many.
    const int64_t lists = (int64_t)c.rows * c.heads;
    const int64_t each = std::min<int64_t>((pl.most + MOVES - 1) / MOVES, MOST_ITEMS / 256 / lists);
    const dim3 moves((unsigned)(lists * each)), threads(256);
    // The rows are read for the last time.  Saying so pays where they are many, and
    // costs where the caches still hold them: with up to 201 MB of them 77 us so and
    // 85 otherwise, with up to 34 MB 55 and 51.
    if (lists * pl.most * 2 * ROW_BYTES > (int64_t)64 << 20)
        hipLaunchKernelGGL((kv_move_kernel<ROW_BYTES, true>), moves, threads, 0, stream, c, a, pl, (int)each);
    else
        hipLaunchKernelGGL((kv_move_kernel<ROW_BYTES, false>), moves, threads, 0, stream, c, a, pl, (int)each);
}

hipError_t launch_kv_evict(const KvCache &c, const KvEvict &a, hipStream_t stream) {
    EvictPlan pl;
    evict_plan(c, a.budget, a.max_len, a.ws, &pl);
    pl.vec = c.cap % 4 == 0 && (((uintptr_t)a.acc | (uintptr_t)a.pos | (uintptr_t)a.acc_out | (uintptr_t)a.pos_out) & 15) == 0;
    const dim3 grid((unsigned)c.rows * c.heads);
    if (!pl.parts) {
        const int n = ranking_threads(a.max_len);
        if (n == 256) hipLaunchKernelGGL((kv_evict_kernel<256, 1>), grid, dim3(n), 0, stream, c, a, pl);
        else if (n == 512) hipLaunchKernelGGL((kv_evict_kernel<512, 2>), grid, dim3(n), 0, stream, c, a, pl);
        else hipLaunchKernelGGL((kv_evict_kernel<1024, 4>), grid, dim3(n), 0, stream, c, a, pl);
    } else {
        const dim3 parts((unsigned)((int64_t)grid.x * pl.parts)), threads(PART_THREADS);
        if (pl.most) {
            hipLaunchKernelGGL(kv_evict_part_kernel<NEWEST>, parts, threads, 0, stream, c, a, pl);
            hipLaunchKernelGGL(kv_evict_part_kernel<COUNT0>, parts, threads, 0, stream, c, a, pl);
            hipLaunchKernelGGL(kv_evict_part_kernel<COUNT1>, parts, threads, 0, stream, c, a, pl);
            hipLaunchKernelGGL(kv_evict_part_kernel<COUNT2>, parts, threads, 0, stream, c, a, pl);
            hipLaunchKernelGGL(kv_evict_part_kernel<TALLY>, parts, threads, 0, stream, c, a, pl);
        }
        hipLaunchKernelGGL(kv_evict_part_kernel<LIST>, parts, threads, 0, stream, c, a, pl);
    }
    if (pl.counts) {
        switch (c.fp8 ? c.dim : 2 * c.dim) {
        case 64: launch_moves<64>(c, a, pl, stream); break;
        case 128: launch_moves<128>(c, a, pl, stream); break;
        case 256: launch_moves<256>(c, a, pl, stream); break;
        default: launch_moves<512>(c, a, pl, stream); break;
        }
    }
    return hipGetLastError();
}

}  // namespace nbw
