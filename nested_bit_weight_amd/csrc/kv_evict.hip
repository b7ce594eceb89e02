// kv_evict.hip -- eviction from the cache by accumulated attention weight,
// gfx950.
//
// For each (row, head) of n > budget slots: the budget largest keys stay, the
// lowest slot first among equals, and the kept rows past the budget move into
// the places below it that became free.  Ranking reads 8 bytes a slot and
// moves copy 4 * dim elements a moved row, so the two are separate problems:
//
//  - Ranking needs a whole (row, head) in one place: one workgroup takes it,
//    with its keys in registers (up to 32 a thread; longer rows are walked in
//    pieces of 32768, their keys in the workspace after the first walk).  The
//    budget-th largest key is found by counting: a histogram of 2048 bins over
//    the 11 bits below the leading bits that all candidates share, the bin that
//    holds the wanted key, and again inside it, until a bin is wanted whole or
//    holds one value.  On attention totals the first two passes do.  Protected
//    slots, which all share the key +infinity, are only counted.  (Bins over
//    fixed leading bits put most totals, alike in sign and exponent, into a few
//    bins, whose atomics then wait for each other.)
//    A slot's place in the list of gaps (below the budget, not kept) or movers
//    (past it, kept) is the number of them in lower slots: ballots within a
//    wave, and one running sum over the waves' counts.
//  - Moves need the whole device: with more than a few a second launch makes
//    them, 64 to a workgroup.  In the steady state of one token over the
//    budget the ranking's workgroup makes its one move itself.
//
// A move reads at or past the budget and writes below it, so moves never meet,
// and no buffer that the ranking reads is written.
#include <algorithm>

#include "kv.h"

namespace nbw {

typedef float f32x4_ev __attribute__((ext_vector_type(4)));
typedef int32_t i32x4_ev __attribute__((ext_vector_type(4)));

constexpr int EVICT_BINS_LOG2 = 11, EVICT_BINS = 1 << EVICT_BINS_LOG2;
constexpr uint32_t KEY_INF = 0xFF800000u, KEY_NEG_INF = 0x007FFFFFu;
constexpr int EVICT_STEP = 32768;   // slots that one walk of the largest kernel holds
constexpr int MOVES = 64;           // moves of a workgroup of the second launch
constexpr int FUSED_MOVES = 16;     // up to so many the ranking's workgroup makes itself

// The workspace: keys of long rows, the lists of each (row, head), their lengths.
struct EvictPlan {
    uint32_t *keys;   // [rows * heads][key_ld], or null
    int64_t key_ld;
    int32_t *lists;   // [rows * heads][2][most]: places to move to, slots to move from
    int most;
    int32_t *counts;  // [rows * heads], or null where the ranking's workgroup moves
    int vec;          // totals and positions may be read 16 bytes at a time
};

// Keys as unsigned numbers of the same order.  -0 and +0 are equal.
__device__ __forceinline__ uint32_t evict_key(float acc, int32_t pos, int32_t newest, const KvEvict &a) {
    if (pos < a.sink || (int64_t)pos > (int64_t)newest - a.recent) return KEY_INF;
    if (acc != acc) return KEY_NEG_INF;
    const uint32_t u = __float_as_uint(acc == 0.f ? 0.f : acc);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// `count` moves of one (row, head): the 16-byte pieces of each move's key and
// value, and its total and position.
template <int ROW_BYTES, int THREADS>
__device__ __forceinline__ void make_moves(const KvCache &c, const KvEvict &a, int row, int head, const int32_t *to,
                                           const int32_t *of, int count) {
    constexpr int VECS = ROW_BYTES / 16, AT_ONCE = 4;
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
                k[j] = *reinterpret_cast<const u32x4_kv *>(c.k + at);
                v[j] = *reinterpret_cast<const u32x4_kv *>(c.v + at);
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

template <int THREADS, int GROUPS>
__global__ __launch_bounds__(THREADS) void kv_evict_kernel(KvCache c, KvEvict a, EvictPlan pl) {
    constexpr int WAVES = THREADS / 64, STEP = THREADS * GROUPS * 4;
    constexpr int TAB = GROUPS * WAVES;  // the waves' counts of one walk, in the order of the slots
    __shared__ int hist[EVICT_BINS];
    __shared__ int red[3][WAVES];
    __shared__ int tab[2][TAB + 1];
    __shared__ int found[3];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int row = blockIdx.x / c.heads, head = blockIdx.x % c.heads;
    const int n = kv_len(a.lens, row, a.max_len), b = a.budget;
    const int64_t base = (int64_t)blockIdx.x * c.cap;
    const float *acc = a.acc + base;
    const int32_t *pos = a.pos + base;
    float *acc_out = a.acc_out + base;
    int32_t *pos_out = a.pos_out + base;
    if (head == 0 && tid == 0) a.lens_out[row] = n < b ? n : b;
    if (pl.counts && tid == 0 && n <= b) pl.counts[blockIdx.x] = 0;

    // Four slots from j on (j a multiple of 4) of a tensor, those past the end as `none`.
    auto four = [&](const auto *p, int j, int end, auto none) {
        decltype(none) x[4] = {none, none, none, none};
        if (pl.vec && j + 4 <= end) {
            typedef decltype(none) vec_t __attribute__((ext_vector_type(4)));
            const vec_t w = *reinterpret_cast<const vec_t *>(p + j);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = w[e];
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < end) x[e] = p[j + e];
        }
        struct R { decltype(none) v[4]; } r;
#pragma unroll
        for (int e = 0; e < 4; ++e) r.v[e] = x[e];
        return r;
    };
    // The first `end` totals and positions from slot j on to the outputs.
    auto copy_out = [&](int j, int end) {
        if (j >= end) return;
        const auto x = four(acc, j, end, 0.f);
        const auto y = four(pos, j, end, 0);
        if (pl.vec && j + 4 <= end) {
            *reinterpret_cast<f32x4_ev *>(acc_out + j) = f32x4_ev{x.v[0], x.v[1], x.v[2], x.v[3]};
            *reinterpret_cast<i32x4_ev *>(pos_out + j) = i32x4_ev{y.v[0], y.v[1], y.v[2], y.v[3]};
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (j + e < end) {
                    acc_out[j + e] = x.v[e];
                    pos_out[j + e] = y.v[e];
                }
        }
    };
    if (n <= b) {
        for (int j = tid * 4; j < n; j += THREADS * 4) copy_out(j, n);
        return;
    }

    const int walks = (n + STEP - 1) / STEP;  // 1 but for rows longer than the largest kernel holds
    uint32_t key[GROUPS][4];
    auto slot_of = [&](int walk, int g) { return walk * STEP + (g * THREADS + tid) * 4; };
    uint32_t *stored = pl.keys ? pl.keys + (int64_t)blockIdx.x * pl.key_ld : nullptr;
    auto get_keys = [&](int walk) {  // of a later walk over a long row
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const int j = slot_of(walk, g);
            const i32x4_ev w = j < n ? *reinterpret_cast<const i32x4_ev *>(stored + j) : i32x4_ev{0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 4; ++e) key[g][e] = (uint32_t)w[e];
        }
    };

    // The newest position, then the keys; how many are +infinity and the range of the rest.
    int32_t newest = INT32_MIN;
    int inf = 0;
    uint32_t lo = 0xFFFFFFFFu, hi = 0;
    {
        float x[GROUPS][4];
        int32_t y[GROUPS][4];
        auto get = [&](int walk, bool totals) {
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                const int j = slot_of(walk, g);
                const auto p = four(pos, j, n, INT32_MIN);
#pragma unroll
                for (int e = 0; e < 4; ++e) y[g][e] = p.v[e];
            }
            if (totals)
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    const auto p = four(acc, slot_of(walk, g), n, 0.f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[g][e] = p.v[e];
                }
        };
        for (int walk = 0; walk < walks; ++walk) {
            get(walk, walks == 1);
#pragma unroll
            for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                for (int e = 0; e < 4; ++e) newest = max(newest, y[g][e]);
        }
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) newest = max(newest, __shfl_xor(newest, d));
        if (lane == 0) red[0][wave] = newest;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w) newest = max(newest, red[0][w]);
        for (int walk = 0; walk < walks; ++walk) {
            if (walks > 1) get(walk, true);
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                const int j = slot_of(walk, g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool there = j + e < n;
                    const uint32_t k = there ? evict_key(x[g][e], y[g][e], newest, a) : 0;  // 0: below every key
                    key[g][e] = k;
                    inf += k == KEY_INF;
                    if (there && k != KEY_INF) {
                        lo = min(lo, k);
                        hi = max(hi, k);
                    }
                }
                if (walks > 1 && j < n)
                    *reinterpret_cast<i32x4_ev *>(stored + j) =
                        i32x4_ev{(int)key[g][0], (int)key[g][1], (int)key[g][2], (int)key[g][3]};
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        inf += __shfl_xor(inf, d);
        lo = min(lo, (uint32_t)__shfl_xor((int)lo, d));
        hi = max(hi, (uint32_t)__shfl_xor((int)hi, d));
    }
    if (lane == 0) {
        red[0][wave] = inf;
        red[1][wave] = (int)lo;
        red[2][wave] = (int)hi;
    }
    __syncthreads();
    inf = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
        inf += red[0][w];
        lo = min(lo, (uint32_t)red[1][w]);
        hi = max(hi, (uint32_t)red[2][w]);
    }

    // All keys above `limit` stay, and of the equals the first `want`; with `all`, every equal.
    uint32_t limit = KEY_INF;
    int want = b;
    bool all = inf == b;
    if (inf < b) {
        want = b - inf;
        for (;;) {  // the want-th largest of the keys within [lo, hi]
            const int bits = lo == hi ? 0 : 32 - __builtin_clz(lo ^ hi);
            if (bits == 0) {
                limit = lo;
                break;
            }
            const int shift = bits > EVICT_BINS_LOG2 ? bits - EVICT_BINS_LOG2 : 0;
            for (int i = tid; i < EVICT_BINS; i += THREADS) hist[i] = 0;
            __syncthreads();
            for (int walk = 0; walk < walks; ++walk) {
                if (walks > 1) get_keys(walk);
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t k = key[g][e];
                        if (k >= lo && k <= hi) atomicAdd(&hist[(k >> shift) & (EVICT_BINS - 1)], 1);
                    }
            }
            __syncthreads();
            // Bins from the top: this thread's are PER of them below tid * PER others.
            constexpr int PER = EVICT_BINS / THREADS;
            int mine = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) mine += hist[EVICT_BINS - 1 - (tid * PER + i)];
            int upto = mine;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int x = __shfl_up(upto, d);
                if (lane >= d) upto += x;
            }
            if (lane == 63) red[0][wave] = upto;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WAVES; ++w)
                if (w < wave) upto += red[0][w];
            int above = upto - mine;
            if (above < want && want <= upto) {
                for (int i = 0; i < PER; ++i) {
                    const int bin = EVICT_BINS - 1 - (tid * PER + i);
                    if (want <= above + hist[bin]) {
                        found[0] = bin;
                        found[1] = above;
                        found[2] = hist[bin];
                        break;
                    }
                    above += hist[bin];
                }
            }
            __syncthreads();
            const uint32_t low = (uint32_t)(((uint64_t)(hi >> shift) & ~(uint64_t)(EVICT_BINS - 1)) | (uint32_t)found[0]) << shift;
            const uint32_t high = low + ((1u << shift) - 1);
            want -= found[1];
            const bool whole = found[2] == want;
            lo = max(lo, low);
            hi = min(hi, high);
            if (whole || shift == 0) {
                limit = lo;
                all = whole;
                break;
            }
            __syncthreads();  // found and hist are free
        }
    }

    // Gaps and movers.
    int32_t *to = pl.lists + (int64_t)blockIdx.x * 2 * pl.most, *of = to + pl.most;
    const uint64_t lower = (1ull << lane) - 1;
    // The running sums over `tab`: entry i becomes the sum of those before it, the last one the total.
    auto sums = [&]() {
        __syncthreads();
        if (wave < 2) {
            int carry = 0;
#pragma unroll
            for (int i0 = 0; i0 < TAB; i0 += 64) {
                const int i = i0 + lane, x = i < TAB ? tab[wave][i] : 0;
                int s = x;
#pragma unroll
                for (int d = 1; d < 64; d <<= 1) {
                    const int up = __shfl_up(s, d);
                    if (lane >= d) s += up;
                }
                if (i < TAB) tab[wave][i] = carry + s - x;
                carry += __shfl(s, 63);
            }
            if (lane == 0) tab[wave][TAB] = carry;
        }
        __syncthreads();
    };
    int equals = 0, gaps = 0, movers = 0;
    for (int walk = 0; walk < walks; ++walk) {
        if (walks > 1) get_keys(walk);
        uint32_t keep = 0;  // bit 4 g + e
#pragma unroll
        for (int g = 0; g < GROUPS; ++g)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                keep |= (uint32_t)(key[g][e] > limit || (all && key[g][e] == limit)) << (4 * g + e);
        if (!all) {
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                int count = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) count += __popcll(__ballot(key[g][e] == limit));
                if (lane == 0) tab[0][g * WAVES + wave] = tab[1][g * WAVES + wave] = count;
            }
            sums();
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                int r = equals + tab[0][g * WAVES + wave];
#pragma unroll
                for (int e = 0; e < 4; ++e) r += __popcll(__ballot(key[g][e] == limit) & lower);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (key[g][e] == limit) keep |= (uint32_t)(r++ < want) << (4 * g + e);
            }
            equals += tab[0][TAB];
            __syncthreads();
        }
        auto is_gap = [&](int g, int e) { return !(keep >> (4 * g + e) & 1) && slot_of(walk, g) + e < b; };
        auto is_mover = [&](int g, int e) { return (keep >> (4 * g + e) & 1) && slot_of(walk, g) + e >= b; };
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
            const int j = slot_of(walk, g);
            int rg = gaps + tab[0][g * WAVES + wave], rm = movers + tab[1][g * WAVES + wave];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                rg += __popcll(__ballot(is_gap(g, e)) & lower);
                rm += __popcll(__ballot(is_mover(g, e)) & lower);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (is_gap(g, e)) to[rg++] = j + e;
                if (is_mover(g, e)) of[rm++] = j + e;
            }
            copy_out(j, b);  // gaps' entries too: their movers overwrite them
        }
        gaps += tab[0][TAB];
        movers += tab[1][TAB];
        __syncthreads();
    }
    if (pl.counts) {
        if (tid == 0) pl.counts[blockIdx.x] = movers;
        return;
    }
    switch (c.fp8 ? c.dim : 2 * c.dim) {
    case 64: make_moves<64, THREADS>(c, a, row, head, to, of, movers); break;
    case 128: make_moves<128, THREADS>(c, a, row, head, to, of, movers); break;
    case 256: make_moves<256, THREADS>(c, a, row, head, to, of, movers); break;
    default: make_moves<512, THREADS>(c, a, row, head, to, of, movers); break;
    }
}

template <int ROW_BYTES>
__global__ __launch_bounds__(256) void kv_move_kernel(KvCache c, KvEvict a, EvictPlan pl, int parts) {
    const int which = blockIdx.x / parts, first = blockIdx.x % parts * MOVES;
    const int count = pl.counts[which];
    if (first >= count) return;
    const int32_t *to = pl.lists + (int64_t)which * 2 * pl.most;
    make_moves<ROW_BYTES, 256>(c, a, which / c.heads, which % c.heads, to + first, to + pl.most + first,
                               min(MOVES, count - first));
}

static int64_t evict_plan(const KvCache &c, int budget, int max_len, uint8_t *base, EvictPlan *pl) {  // -1: too many workgroups
    const int64_t lists = (int64_t)c.rows * c.heads;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        uint8_t *p = base ? base + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    pl->most = std::max(0, std::min(budget, max_len - budget));
    pl->keys = nullptr;
    pl->key_ld = (max_len + 3) / 4 * 4;
    pl->counts = nullptr;
    pl->lists = nullptr;
    if (pl->most == 0) return 0;  // no row is over the budget
    if (lists * ((pl->most + MOVES - 1) / MOVES) > INT32_MAX) return -1;
    pl->lists = (int32_t *)take(lists * 2 * pl->most * 4);
    if (pl->most > FUSED_MOVES) pl->counts = (int32_t *)take(lists * 4);
    if (max_len > EVICT_STEP) pl->keys = (uint32_t *)take(lists * pl->key_ld * 4);
    return at;
}

int64_t kv_evict_workspace_bytes(const KvCache &c, int budget, int max_len) {
    EvictPlan pl;
    return evict_plan(c, budget, max_len, nullptr, &pl);
}

hipError_t launch_kv_evict(const KvCache &c, const KvEvict &a, hipStream_t stream) {
    EvictPlan pl;
    evict_plan(c, a.budget, a.max_len, a.ws, &pl);
    pl.vec = c.cap % 4 == 0 && (((uintptr_t)a.acc | (uintptr_t)a.pos | (uintptr_t)a.acc_out | (uintptr_t)a.pos_out) & 15) == 0;
    const dim3 grid((unsigned)c.rows * c.heads);
    // The smallest workgroup that holds the longest row's keys in its registers.
    if (a.max_len <= 1024) hipLaunchKernelGGL((kv_evict_kernel<256, 1>), grid, dim3(256), 0, stream, c, a, pl);
    else if (a.max_len <= 4096) hipLaunchKernelGGL((kv_evict_kernel<1024, 1>), grid, dim3(1024), 0, stream, c, a, pl);
    else if (a.max_len <= 16384) hipLaunchKernelGGL((kv_evict_kernel<1024, 4>), grid, dim3(1024), 0, stream, c, a, pl);
    else hipLaunchKernelGGL((kv_evict_kernel<1024, 8>), grid, dim3(1024), 0, stream, c, a, pl);
    if (pl.counts) {
        const int parts = (pl.most + MOVES - 1) / MOVES;
        const dim3 moves((unsigned)((int64_t)grid.x * parts));
        switch (c.fp8 ? c.dim : 2 * c.dim) {
        case 64: hipLaunchKernelGGL(kv_move_kernel<64>, moves, dim3(256), 0, stream, c, a, pl, parts); break;
        case 128: hipLaunchKernelGGL(kv_move_kernel<128>, moves, dim3(256), 0, stream, c, a, pl, parts); break;
        case 256: hipLaunchKernelGGL(kv_move_kernel<256>, moves, dim3(256), 0, stream, c, a, pl, parts); break;
        default: hipLaunchKernelGGL(kv_move_kernel<512>, moves, dim3(256), 0, stream, c, a, pl, parts); break;
        }
    }
    return hipGetLastError();
}

}  // namespace nbw
