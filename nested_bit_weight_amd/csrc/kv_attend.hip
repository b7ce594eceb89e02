// kv_attend.hip -- attention of one new token for each row over its cached
// ones, gfx950.
//
// For a query head g and the n slots of its row
//     s_j = scale q.k_j,   o = sum_j 2^(s_j' - m) v_j / sum_j 2^(s_j' - m),
// s' = s log2(e), with any m near the largest s'.  Every key and value is read
// once and meets the G = q_heads / heads query heads of its head, 4 G flops for
// 4 bytes (2 in the 8-bit cache): at the usual G = 4..8 the operator is bound
// by the bandwidth of memory by a wide margin, and what follows is arranged
// around keeping loads in flight.
//
// Work: units of CHUNK = 128 slots of one (row, head) in the order (row, head,
// chunk), divided among as many workgroups as the device holds at once, whatever
// the rows' lengths are: one long row is spread over the whole device, many short
// ones are packed.  The lengths stay on the device; each workgroup finds its units
// from their running sum.  A run of units within one (row, head) is a piece; a
// (row, head) that is one piece is finished there, others leave their parts (m,
// sum, o) in the workspace, which a second launch joins in a fixed order.
//
// A piece: wave w takes the 32-slot tile w of each unit, everything in its
// registers, with the next tile's keys and values loading while this one's are
// used.  S^T = K Q^T and O = P V on v_mfma_f32_16x16x32_bf16:
//  - A of the first product is 16 keys by 32 dims, loaded as it is used: lane
//    l holds 16 bytes of key l % 16.  Its result has head l % 16 in lane l and
//    slots 4 (l / 16) + 0..3 in the lane's four registers, of each half tile;
//  - these are the rows of P that the second product's A operand wants in that
//    lane, if slot 4 (l / 16) + i of half h is given the product's inner index
//    8 (l / 16) + 4 h + i: P never leaves the lane;
//  - V is loaded row by row, lane l the dims 8 (l % 16) .. + 7 of the eight
//    slots of its quarter, and one v_perm for each pair of slots makes the B
//    operand of column t: dim 8 (l % 16) + t.
// The weights enter the second product as three bf16 parts, which hold all 24 bits of
// them; sums of p are taken in fp32 before that.  With up to 8 heads the two upper parts
// share one product, in its rows 0..7 and 8..15, whose scores are computed twice instead
// of rows standing empty, and half of the lowest part is in each half of another.  (With two
// parts, 16 bits, everything takes as long within 1%: 64 rows 201 us, 24 rows with 12
// heads 49, one row of 333 slots 7.6 and 7.8 so.)
//
// Measured (128 dims, 8 heads): 64 rows of up to 8192 slots, 1.2 GB: 200 us, 6.0 TB/s
// (a plain read of as much: 175 us), with totals 248; one row of 131071 slots, 537 MB,
// 64 query heads: 88 us, 6.1 TB/s; 16 rows of up to 2048 slots: 15 us, half of it the
// chain of loads before the first key and the join; one row of 333 slots: 7 us.
//
// The running maximum m of a head is only raised, and o and the sum rescaled,
// when a score passes it by more than 8 (a factor of 2^8): the check is one
// comparison and a branch that is almost never taken after the first tile.
#include <algorithm>

#include "kv.h"

namespace nbw {

typedef float f32x4_kv __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_kv __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_kv __attribute__((ext_vector_type(2)));

constexpr int ATTEND_WAVES = 4;
constexpr int ATTEND_THREADS = 64 * ATTEND_WAVES;
constexpr int TILE = 32;                     // slots of one wave's step
constexpr int CHUNK = TILE * ATTEND_WAVES;   // slots of a unit
constexpr float RAISE = 8.f;                 // how far a score may pass the running maximum
constexpr float TINY = 1.17549435e-38f;      // the smallest normal number, fp32's and bf16's

#define NEG_INF (-__builtin_inff())

// A word that no kernel of this launch writes, at an address all lanes share: a
// scalar load, which does not wait in line behind the keys and values in flight.
__device__ __forceinline__ int32_t uniform_word(const int32_t *p) {
    return *reinterpret_cast<const __attribute__((address_space(4))) int32_t *>(reinterpret_cast<uintptr_t>(p));
}

// The wave's accesses to LDS before this are over, in all lanes, before those after it.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The launch's division of work and its scratch, the same for both kernels.
struct AttendPlan {
    int wgs;             // workgroups of the first launch
    int group;           // query heads of a head
    int blocks;          // blocks of up to 16 query heads that a head's are taken in
    int block_heads;     // query heads of a block (the last may have fewer)
    int undivided;       // every (row, head, block) has a workgroup of its own
    int32_t *before;     // [rows + 1] units of one (head, block) before each row
    int32_t *pieces;     // [rows + 1] pieces of one (head, block) before each row, then their units
    float *whole;        // [rows][heads * blocks][16][2]: m and sum where one workgroup had it all
    float *part_ml;      // [2 * wgs][16][2]: m and sum of a piece
    float *part_o;       // [2 * wgs][block_heads][dim]
    float *scores;       // [unit][wave][half][quarter][block_heads][4], with totals only
    int sharers;         // workgroups that add to the totals
    int vec;             // totals may be read and written 16 bytes at a time
};

// Weights are up to 2^RAISE, and n of them meet the values.  Times this power of two they
// sum to 1 at the most, and finite values cannot run over.
__device__ __forceinline__ float weights_by(int n) {
    return __uint_as_float((uint32_t)(127 - (int)RAISE - (n > 1 ? 32 - __builtin_clz(n - 1) : 0)) << 23);
}

// The workgroup whose share a unit is in.
__device__ __forceinline__ int owner_of(int64_t unit, int64_t units, int shares) {
    return (int)(((unit + 1) * shares - 1) / units);
}

// The parts of one (row, head, block): n of them, part i at place(i).  With equal
// shares workgroup w leaves what began in an earlier share at place 2 w, and what
// begins in its own and goes on past it at 2 w + 1; pieces of equal length are at
// twice their number.
struct Parts {
    int n, first, odd;
    __device__ __forceinline__ int place(int i) const { return 2 * (first + i) + (i == 0 ? odd : 0); }
};
__device__ __forceinline__ Parts parts_of(const KvCache &c, const AttendPlan &pl, int row, int vh, int at, int chunks) {
    const int vheads = c.heads * pl.blocks, k = pl.pieces[c.rows + 1];
    if (k) {
        const int n = (chunks + k - 1) / k;
        return {n, pl.pieces[row] * vheads + vh * n, 0};
    }
    const int64_t units = (int64_t)pl.before[c.rows] * vheads, seg0 = (int64_t)at * vheads + (int64_t)vh * chunks;
    const int shares = (int)min((int64_t)pl.wgs, units);
    const int w0 = owner_of(seg0, units, shares);
    return {owner_of(seg0 + chunks - 1, units, shares) - w0 + 1, w0, 1};
}

// Scores that a wave holds back (what leaves two workgroups room on a CU), and
// their tiles: 12 of eight heads, 5 of sixteen.
__host__ __device__ constexpr int held_scores(bool pack) { return pack ? 12 * TILE * 8 : 5 * TILE * 16; }
__host__ __device__ constexpr int most_held(int block_heads) { return held_scores(block_heads <= 8) / (TILE * block_heads); }

// One wave's tile: keys and values as loaded, and which slots count.
template <int DIM, bool FP8>
struct Tile {
    static constexpr int KV4 = FP8 ? DIM / 64 : DIM / 32;  // 16-byte loads of a key
    static constexpr int NC = DIM > 128 ? DIM / 128 : 1;   // blocks of dims of a value
    static constexpr int DPL = DIM / NC / 16;              // dims of a block in one lane
    static constexpr int VW = FP8 ? DPL / 4 : DPL / 2;     // words of them
    u32x4_kv k[2][KV4];
    uint32_t v[2][4][NC][VW];
    uint32_t there;  // bit 4 h + i: slot 4 (lane / 16) + i of half h
};

template <bool NT, class V>
__device__ __forceinline__ V load_as(const uint8_t *p) {
    if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const V *>(p));
    else return *reinterpret_cast<const V *>(p);
}

template <bool NT, int W>
__device__ __forceinline__ void load_words(uint32_t *out, const uint8_t *p) {
    if constexpr (W == 4) {
        const u32x4_kv x = load_as<NT, u32x4_kv>(p);
        out[0] = x[0], out[1] = x[1], out[2] = x[2], out[3] = x[3];
    } else if constexpr (W == 2) {
        const u32x2_kv x = load_as<NT, u32x2_kv>(p);
        out[0] = x[0], out[1] = x[1];
    } else {
        out[0] = load_as<NT, uint32_t>(p);
    }
}

// Two 8-bit values of a word (half 0: its lower two) as a pair of bf16, exact.
template <int HALF>
__device__ __forceinline__ uint32_t fp8_pair(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HALF));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    const bf16x2_kv p = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, p);
}

// acc_out = decay * acc + w for slots slot .. slot + 3 below n of the (row, head) at `base`.
__device__ __forceinline__ void add_totals(const KvAttend &a, int64_t base, int slot, int n, f32x4_kv w, bool vec) {
    const float *acc = a.acc + base + slot;
    float *out = a.acc_out + base + slot;
    if (vec && slot + 4 <= n) {
        const f32x4_kv was = *reinterpret_cast<const f32x4_kv *>(acc);
        *reinterpret_cast<f32x4_kv *>(out) = was * a.decay + w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (slot + e < n) out[e] = a.decay * acc[e] + w[e];
    }
}

template <int DIM, bool FP8, bool PACK, bool SMALL, bool NT, bool WEIGHTS>
__global__ __launch_bounds__(ATTEND_THREADS, DIM > 128 ? 1 : 2) void kv_attend_kernel(KvCache c, KvAttend a, AttendPlan pl) {
    using T = Tile<DIM, FP8>;
    constexpr int HR = PACK ? 8 : 16;                 // heads a workgroup holds
    constexpr int ROW_BYTES = FP8 ? DIM : DIM * 2;
    constexpr int COLS = DIM / T::NC;                 // dims of a block
    constexpr int QF = DIM / 32;                      // Q operands
    __shared__ int scan[ATTEND_WAVES];
    __shared__ int found[2];
    __shared__ __align__(16) float wave_m[HR][ATTEND_WAVES], wave_l[HR][ATTEND_WAVES];
    __shared__ float head_ml[HR][2];
    // Each wave's results at the end of a piece and, with totals, the scores of its
    // last tiles.
    constexpr int HELD = WEIGHTS ? held_scores(PACK) : 0, POOL = HELD + HR * COLS;  // a wave's
    __shared__ __align__(16) float pool[ATTEND_WAVES * POOL];
    auto wave_o = [&](int w, int h, int d) -> float * { return pool + w * POOL + HELD + h * COLS + d; };
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int quad = lane >> 4, col = lane & 15;
    const int vheads = c.heads * pl.blocks;

    auto chunks_of = [&](int n) { return (n + CHUNK - 1) / CHUNK; };
    auto zeros = [&](int row, int from, int to) {  // query heads from .. to - 1 of a row without a slot
        for (int i = from * DIM / 8 + tid; i < to * DIM / 8; i += ATTEND_THREADS)
            reinterpret_cast<u32x4_kv *>(a.out + (int64_t)row * a.out_ld)[i] = u32x4_kv{0, 0, 0, 0};
    };

    // This workgroup's first piece, and with equal shares its units [u, u1).
    int row, row_at = 0, len, row_chunks, vh, c0, c1, part = 0, u = 0, u1 = 0;
    int32_t early[4];
    if (pl.undivided) {
        row = blockIdx.x / vheads;
        vh = blockIdx.x % vheads;
        len = uniform_word(a.lens + row);
        if (!SMALL) {  // the first page numbers are asked for along with the length
            const int32_t *table = c.table + (int64_t)row * c.table_ld;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                early[i] = uniform_word(table + (min(i / 2 * CHUNK + wave * TILE + i % 2 * 16, c.cap - 1) >> c.page_log2));
            asm volatile("" : "+s"(len), "+s"(early[0]), "+s"(early[1]), "+s"(early[2]), "+s"(early[3]));
        }
        len = min(max(len, 0), a.max_len);
        row_chunks = chunks_of(len);
        c0 = 0;
        c1 = row_chunks;
        if (len == 0) {
            const int from = vh / pl.blocks * pl.group + vh % pl.blocks * pl.block_heads;
            zeros(row, from, from + min(pl.block_heads, pl.group - vh % pl.blocks * pl.block_heads));
            return;
        }
    } else {
        // Units of one (head, block) before this workgroup's rows.  Up to 64 rows: lane
        // r of every wave has row r, and no wave waits for another.  More: strips of
        // rows for each thread, summed over the workgroup.
        const bool few = c.rows <= 64;
        const int strip = few ? 1 : (c.rows + ATTEND_THREADS - 1) / ATTEND_THREADS;
        const int r0 = few ? lane : tid * strip, r1 = min(r0 + strip, c.rows);
        int mine = 0, first_len = 0;
        if (few) {
            if (r0 < r1) first_len = kv_len(a.lens, r0, a.max_len);
            mine = chunks_of(first_len);
        } else {
            for (int r = r0; r < r1; ++r) mine += chunks_of(kv_len(a.lens, r, a.max_len));
        }
        int upto = wave_running_sum(mine), chunks = __builtin_amdgcn_readlane(upto, 63);
        if (!few) {
            if (lane == 63) scan[wave] = upto;
            __syncthreads();
            chunks = 0;
#pragma unroll
            for (int w = 0; w < ATTEND_WAVES; ++w) {
                if (w < wave) upto += scan[w];
                chunks += scan[w];
            }
        }
        const int before = upto - mine;
        const int64_t units = (int64_t)chunks * vheads;

        // Pieces of k units each, one for a workgroup, if k need be little more than an
        // equal share: a share that runs over from one (row, head) into the next costs
        // its workgroup a second start, about as long as a unit takes.
        int k = 0, pieces = 0;
        if (few && units) {
            const int share = (int)((units + pl.wgs - 1) / pl.wgs);
            for (int t = share; t <= share + 1 && !k; ++t) {
                pieces = wave_running_sum((mine + t - 1) / t);
                if ((int64_t)__builtin_amdgcn_readlane(pieces, 63) * vheads <= pl.wgs) k = t;
            }
        }
        if (blockIdx.x == 0 && (!few || wave == 0)) {
            int at = before;
            for (int r = r0; r < r1; ++r) {
                pl.before[r] = at;
                if (few) pl.pieces[r] = k ? pieces - (mine + k - 1) / k : 0;
                else at += chunks_of(kv_len(a.lens, r, a.max_len));
            }
            if (tid == 0) {
                pl.before[c.rows] = chunks;
                pl.pieces[c.rows + 1] = k;
            }
        }
        for (int r = blockIdx.x; r < c.rows; r += pl.wgs)
            if ((few ? __builtin_amdgcn_readlane(first_len, r) : kv_len(a.lens, r, a.max_len)) == 0) zeros(r, 0, a.q_heads);
        if (k) {
            const int mine_k = (mine + k - 1) / k;
            const unsigned long long at = __ballot((int)blockIdx.x < pieces * vheads);
            if (!at) return;
            row = __builtin_ctzll(at);
            row_at = __builtin_amdgcn_readlane(before, row);
            len = __builtin_amdgcn_readlane(first_len, row);
            row_chunks = chunks_of(len);
            const int n = __builtin_amdgcn_readlane(mine_k, row);
            const int in = (int)blockIdx.x - (__builtin_amdgcn_readlane(pieces, row) - n) * vheads;
            vh = in / n;
            c0 = in % n * k;
            c1 = min(c0 + k, row_chunks);
            part = 2 * blockIdx.x;
        } else {
            const int shares = (int)min((int64_t)pl.wgs, units);  // none is empty
            if ((int)blockIdx.x >= shares) return;
            u = (int)(units * blockIdx.x / shares);
            u1 = (int)(units * (blockIdx.x + 1) / shares);
            const bool here = (int64_t)before * vheads <= u && u < (int64_t)upto * vheads;
            if (few) {
                row = __builtin_ctzll(__ballot(here));
                row_at = __builtin_amdgcn_readlane(before, row);
                len = __builtin_amdgcn_readlane(first_len, row);
            } else {
                if (here) {
                    int at = before, r = r0;
                    for (;; ++r) {
                        const int n = chunks_of(kv_len(a.lens, r, a.max_len));
                        if (u < (int64_t)(at + n) * vheads) break;
                        at += n;
                    }
                    found[0] = r;
                    found[1] = at;
                }
                __syncthreads();
                row = __builtin_amdgcn_readfirstlane(found[0]);
                row_at = __builtin_amdgcn_readfirstlane(found[1]);
                len = __builtin_amdgcn_readfirstlane(kv_len(a.lens, row, a.max_len));
            }
            row_chunks = chunks_of(len);
            vh = (u - row_at * vheads) / row_chunks;
            c0 = u - row_at * vheads - vh * row_chunks;
            c1 = min(row_chunks, c0 + u1 - u);
            part = 2 * blockIdx.x + (c0 == 0);
        }
    }

    for (;;) {  // the piece: chunks [c0, c1) of (row, vh)
        const int64_t seg0 = (int64_t)row_at * vheads + vh * row_chunks;  // its first unit
        const int head = vh / pl.blocks, block = vh % pl.blocks;
        const int g0 = block * pl.block_heads, heads = min(pl.block_heads, pl.group - g0);
        const int32_t *table = c.table + (int64_t)row * c.table_ld;
        const float down = weights_by(len);
        const float by = a.scale * 1.44269504088896340736f * (FP8 ? c.k_scale[head] : 1.f), v_by = FP8 ? c.v_scale[head] : 1.f;

        // Q as the first product's B operand: column `col`'s head, the dims that
        // the key operand of the same number holds in this lane.
        u32x4_kv qf[QF];
        const int qh = PACK ? col & 7 : col;
        {
            const uint16_t *q = a.q + (int64_t)row * a.q_ld + ((int64_t)head * pl.group + g0 + (qh < heads ? qh : 0)) * DIM;
#pragma unroll
            for (int f = 0; f < QF; ++f) {
                const int d = FP8 ? (f >> 1) * 64 + quad * 16 + (f & 1) * 8 : f * 32 + quad * 8;
                qf[f] = qh < heads ? *reinterpret_cast<const u32x4_kv *>(q + d) : u32x4_kv{0, 0, 0, 0};
            }
        }

        // Page numbers of a chunk's tile.  Pages of 16 slots and more: one for each
        // half, the same in all lanes; smaller ones: lane l has slot l % 32's.  Past the
        // row's length they are whatever the table holds; in their place, and for pages
        // that are not there, the pool's first page is loaded and left out.
        struct Pages { int32_t p[SMALL ? 1 : 2]; };
        auto pages_of = [&](int chunk) {
            Pages r;
            const int slot = chunk * CHUNK + wave * TILE;
            if constexpr (SMALL) {
                const int s = slot + (lane & 31);
                r.p[0] = table[min(s, c.cap - 1) >> c.page_log2];
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    r.p[h] = uniform_word(table + (min(slot + 16 * h, c.cap - 1) >> c.page_log2));
            }
            return r;
        };
        auto load = [&](T &t, const Pages &pg, int chunk) {
            const int slot = chunk * CHUNK + wave * TILE, mask = (1 << c.page_log2) - 1;
            t.there = 0;
            if constexpr (SMALL) {
                const int32_t own = pg.p[0];
                const int mine_ok = own >= 0 && own < c.pages;
                const int32_t safe = mine_ok ? own : -1;
                auto place = [&](int s, bool &ok) -> int64_t {  // byte offset of slot s (0..31) of the tile
                    const int32_t p = __shfl(safe, s);
                    ok = p >= 0 && slot + s < len;
                    return ((((int64_t)(ok ? p : 0) * c.heads + head) << c.page_log2) + ((slot + s) & mask)) * ROW_BYTES;
                };
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    bool ok;
                    const uint8_t *p = c.k + place(16 * h + col, ok) + quad * 16;
#pragma unroll
                    for (int f = 0; f < T::KV4; ++f) t.k[h][f] = load_as<NT, u32x4_kv>(p + f * 64);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint8_t *q = c.v + place(16 * h + quad * 4 + i, ok) + col * T::VW * 4;
                        t.there |= (uint32_t)ok << (4 * h + i);
#pragma unroll
                        for (int n = 0; n < T::NC; ++n) load_words<NT, T::VW>(t.v[h][i][n], q + n * (ROW_BYTES / T::NC));
                    }
                }
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int s = slot + 16 * h;
                    const bool ok = s < len && (uint32_t)pg.p[h] < (uint32_t)c.pages;
                    const int left = ok ? min(len - s, 16) - quad * 4 : 0;
                    t.there |= (left >= 4 ? 15u : left <= 0 ? 0u : (1u << left) - 1) << (4 * h);
                    const int64_t base = ((((int64_t)(ok ? pg.p[h] : 0) * c.heads + head) << c.page_log2) + (s & mask)) * ROW_BYTES;
                    const uint8_t *kb = c.k + base, *vb = c.v + base;
                    const uint32_t ko = col * ROW_BYTES + quad * 16, vo = quad * 4 * ROW_BYTES + col * T::VW * 4;
#pragma unroll
                    for (int f = 0; f < T::KV4; ++f) t.k[h][f] = load_as<NT, u32x4_kv>(kb + ko + f * 64);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int n = 0; n < T::NC; ++n)
                            load_words<NT, T::VW>(t.v[h][i][n], vb + vo + i * ROW_BYTES + n * (ROW_BYTES / T::NC));
                }
            }
        };

        f32x4_kv o[T::NC][T::DPL];
#pragma unroll
        for (int n = 0; n < T::NC; ++n)
#pragma unroll
            for (int t = 0; t < T::DPL; ++t) o[n][t] = f32x4_kv{0.f, 0.f, 0.f, 0.f};
        float m = NEG_INF, sum = 0.f;

        // Scores wait in LDS and leave a few tiles at a time: a store counts among the
        // operations in flight, in order, so that with one in every tile each tile
        // waited for the last one's to reach memory (64 rows, 1.2 GB: 250 us so, 237 held
        // back, 196 without the stores).
        float *scores = pool + wave * POOL;
        const int most_held = nbw::most_held(pl.block_heads);
        int held = 0;
        auto put_scores = [&](int chunk) {  // up to this chunk's
            const int each = TILE / 4 * pl.block_heads;  // 16-byte pieces of a tile
            float *dst = pl.scores + ((seg0 + chunk - held + 1) * ATTEND_WAVES + wave) * each * 4;
            wave_fence();
            for (int i = lane; i < held * each; i += 64)
                *reinterpret_cast<f32x4_kv *>(dst + ((int64_t)(i / each) * ATTEND_WAVES * each + i % each) * 4) =
                    *reinterpret_cast<const f32x4_kv *>(scores + i * 4);
            wave_fence();
            held = 0;
        };
        auto use = [&](T &t, int chunk) {
            f32x4_kv s[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int f = 0; f < QF; ++f)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    u32x4_kv kf;
                    if constexpr (FP8) {
                        const uint32_t w0 = t.k[h][f >> 1][(f & 1) * 2], w1 = t.k[h][f >> 1][(f & 1) * 2 + 1];
                        kf = u32x4_kv{fp8_pair<0>(w0), fp8_pair<1>(w0), fp8_pair<0>(w1), fp8_pair<1>(w1)};
                    } else {
                        kf = t.k[h][f];
                    }
                    s[h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_kv, kf),
                                                                   __builtin_bit_cast(bf16x8_kv, qf[f]), s[h], 0, 0, 0);
                }
            const bool full = __all(t.there == 0xFFu);
            float x[8], top = NEG_INF;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = s[i >> 2][i & 3] * by;
            if (!full) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = t.there >> i & 1 ? x[i] : NEG_INF;
            }
            if constexpr (WEIGHTS) {
                float *dst = scores + held * TILE * pl.block_heads + (quad * pl.block_heads + col) * 4;
                if (col < heads) {
                    *reinterpret_cast<f32x4_kv *>(dst) = f32x4_kv{x[0], x[1], x[2], x[3]};
                    *reinterpret_cast<f32x4_kv *>(dst + 16 * pl.block_heads) = f32x4_kv{x[4], x[5], x[6], x[7]};
                }
                if (++held == most_held && chunk + 1 < c1) put_scores(chunk);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) top = fmaxf(top, x[i]);
            if (__any(top > m + RAISE)) {
                top = fmaxf(m, top);
                top = fmaxf(top, __shfl_xor(top, 16));
                top = fmaxf(top, __shfl_xor(top, 32));
                const float fade = top == m ? 1.f : exp2f(m - top);  // equal: -inf, or nothing to do
                m = top;
                sum *= fade;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float f = __shfl(fade, quad * 4 + i);
#pragma unroll
                    for (int n = 0; n < T::NC; ++n)
#pragma unroll
                        for (int e = 0; e < T::DPL; ++e) o[n][e][i] *= f;
                }
            }
            const float ref = m == NEG_INF ? 0.f : m;
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = __builtin_amdgcn_exp2f(x[i] - ref) * down;
                sum += p[i];
            }
            // The weights' 24 bits as three bf16 parts: each but the last is cut off, not
            // rounded, so that none is negative, and none of a weight's is 0 unless it is, so
            // an infinite value stays one (0 * inf and inf - inf would be NaN).  A weight
            // of 0 adds nothing, however large its value.
            u32x4_kv hi, mid, lo;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a0 = p[2 * i], a1 = p[2 * i + 1], t0 = fminf(a0, TINY), t1 = fminf(a1, TINY);
                hi[i] = __builtin_amdgcn_perm(__float_as_uint(a1), __float_as_uint(a0), 0x07060302u);
                const float b0 = fmaxf(a0 - bf16_lo(hi[i]), t0), b1 = fmaxf(a1 - bf16_hi(hi[i]), t1);
                mid[i] = __builtin_amdgcn_perm(__float_as_uint(b1), __float_as_uint(b0), 0x07060302u);
                constexpr float each = PACK ? 0.5f : 1.f;  // of the lowest part, in how many rows it is
                lo[i] = pack_bf16(fmaxf((b0 - bf16_lo(mid[i])) * each, t0), fmaxf((b1 - bf16_hi(mid[i])) * each, t1));
                if (PACK) hi[i] = col < 8 ? hi[i] : mid[i];
            }
#pragma unroll
            for (int n = 0; n < T::NC; ++n) {
                uint32_t w[8][T::DPL / 2];  // the eight slots' dims as pairs of bf16
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t *src = t.v[i >> 2][i & 3][n];
#pragma unroll
                    for (int d = 0; d < T::DPL / 2; ++d) {
                        if constexpr (FP8) w[i][d] = d & 1 ? fp8_pair<1>(src[d >> 1]) : fp8_pair<0>(src[d >> 1]);
                        else w[i][d] = src[d];
                    }
                }
                if (!full) {  // 0 * what lies there would be NaN for an infinity or a NaN
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int d = 0; d < T::DPL / 2; ++d) w[i][d] = t.there >> i & 1 ? w[i][d] : 0u;
                }
#pragma unroll
                for (int e = 0; e < T::DPL; ++e) {
                    u32x4_kv vf;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        vf[i] = __builtin_amdgcn_perm(w[2 * i + 1][e >> 1], w[2 * i][e >> 1], e & 1 ? 0x07060302u : 0x05040100u);
                    o[n][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_kv, hi),
                                                                      __builtin_bit_cast(bf16x8_kv, vf), o[n][e], 0, 0, 0);
                    if (!PACK)
                        o[n][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_kv, mid),
                                                                          __builtin_bit_cast(bf16x8_kv, vf), o[n][e], 0, 0, 0);
                    o[n][e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_kv, lo),
                                                                      __builtin_bit_cast(bf16x8_kv, vf), o[n][e], 0, 0, 0);
                }
            }
        };

        // Two tiles in turn.  Page numbers are asked for one tile further ahead, and
        // before the tile that they do not belong to: loads return in order, and
        // waiting for them must not mean waiting for that tile.  For the same reason
        // the loop has no load that depends on a condition: how many are in flight
        // when a tile is used is then known, and only its own are waited for.
        {
            T ta, tb;
            Pages pa, pb;
            if (!SMALL && pl.undivided) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    pa.p[h * !SMALL] = early[h];
                    pb.p[h * !SMALL] = early[2 + h];
                }
            } else {
                pa = pages_of(c0);
                pb = pages_of(c0 + 1);
            }
            load(ta, pa, c0);
            int ch = c0;
            for (; ch + 2 < c1; ch += 2) {
                pa = pages_of(ch + 2);
                load(tb, pb, ch + 1);
                use(ta, ch);
                pb = pages_of(ch + 3);
                load(ta, pa, ch + 2);
                use(tb, ch + 1);
            }
            if (ch + 1 < c1) {
                load(tb, pb, ch + 1);
                use(ta, ch);
                use(tb, ch + 1);
            } else {
                use(ta, ch);
            }
        }

        // With all of its row's scores still in LDS a workgroup adds to the totals itself.
        const bool whole = c0 == 0 && c1 == row_chunks;
        const bool totals = WEIGHTS && whole && pl.blocks == 1 && c1 <= most_held;
        if (WEIGHTS && !totals) put_scores(c1 - 1);

        // The four waves' results together: each one's o as it stands, and what to
        // multiply it by.
        sum += __shfl_xor(sum, 16);
        sum += __shfl_xor(sum, 32);
        if (lane < HR) {
            wave_m[lane][wave] = m;
            wave_l[lane][wave] = sum;
        }
        auto put_o = [&](int n) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int h = quad * 4 + i;
                float x[T::DPL];
#pragma unroll
                for (int e = 0; e < T::DPL; ++e) {
                    x[e] = o[n][e][i];
                    if (PACK) {  // rows 8..15, in the upper half of the wave, are the weights' lower parts
                        const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(x[e]), __float_as_uint(x[e]), false, false);
                        x[e] = __uint_as_float(both[0]) + __uint_as_float(both[1]);
                    }
                }
                if (h < HR)
#pragma unroll
                    for (int e = 0; e < T::DPL; e += 4)
                        *reinterpret_cast<f32x4_kv *>(wave_o(wave, h, col * T::DPL + e)) = f32x4_kv{x[e], x[e + 1], x[e + 2], x[e + 3]};
            }
        };
        put_o(0);
        __syncthreads();
        auto merged = [&](int h, f32x4_kv &fade, float &top, float &total) {
            const f32x4_kv mw = *reinterpret_cast<const f32x4_kv *>(wave_m[h]), lw = *reinterpret_cast<const f32x4_kv *>(wave_l[h]);
            top = fmaxf(fmaxf(mw[0], mw[1]), fmaxf(mw[2], mw[3]));
            total = 0.f;
#pragma unroll
            for (int w = 0; w < ATTEND_WAVES; ++w) {
                fade[w] = mw[w] == top ? 1.f : __builtin_amdgcn_exp2f(mw[w] - top);
                total += lw[w] * fade[w];
            }
        };
        if (WEIGHTS || !whole)
            if (tid < heads) {
                f32x4_kv fade;
                float top, total;
                merged(tid, fade, top, total);
                if (!whole) {
                    pl.part_ml[(part * 16 + tid) * 2] = top;
                    pl.part_ml[(part * 16 + tid) * 2 + 1] = total;
                } else if (totals) {
                    head_ml[tid][0] = top == NEG_INF ? 0.f : top;
                    head_ml[tid][1] = total == 0.f ? 0.f : down / total;
                } else {
                    float *w = pl.whole + (((int64_t)row * vheads + vh) * 16 + tid) * 2;
                    w[0] = top;
                    w[1] = total;
                }
            }
#pragma unroll
        for (int n = 0; n < T::NC; ++n) {
            if (n) {
                __syncthreads();
                put_o(n);
                __syncthreads();
            }
            for (int i = tid; i < heads * (COLS / 4); i += ATTEND_THREADS) {
                const int h = i / (COLS / 4), d = i % (COLS / 4) * 4;
                f32x4_kv fade, x = {0.f, 0.f, 0.f, 0.f};
                float top, total;
                merged(h, fade, top, total);
#pragma unroll
                for (int w = 0; w < ATTEND_WAVES; ++w) x += *reinterpret_cast<const f32x4_kv *>(wave_o(w, h, d)) * fade[w];
                if (whole) {
                    const float inv = total == 0.f ? 0.f : v_by / total;
                    if (total == 0.f) x = f32x4_kv{0.f, 0.f, 0.f, 0.f};  // nothing to attend to, whatever the values are
                    uint16_t *dst = a.out + (int64_t)row * a.out_ld + ((int64_t)head * pl.group + g0 + h) * DIM + n * COLS + d;
                    *reinterpret_cast<u32x2_kv *>(dst) = u32x2_kv{pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv)};
                } else {
                    float *dst = pl.part_o + ((int64_t)part * pl.block_heads + h) * DIM + n * COLS + d;
                    *reinterpret_cast<f32x4_kv *>(dst) = x;
                }
            }
        }
        if (totals) {
            __syncthreads();
            const int64_t base = ((int64_t)row * c.heads + head) * c.cap;
            for (int i = lane; i < c1 * 8; i += 64) {  // four slots of this wave's tiles
                const int slot = i / 8 * CHUNK + wave * TILE + i % 8 * 4;
                if (slot >= len) continue;
                const float *s = scores + i * 4 * pl.block_heads;
                f32x4_kv w = {0.f, 0.f, 0.f, 0.f};
                for (int h = 0; h < heads; ++h) {
                    const f32x4_kv x = *reinterpret_cast<const f32x4_kv *>(s + h * 4);
                    const float hm = head_ml[h][0], hi = head_ml[h][1];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] += __builtin_amdgcn_exp2f(x[e] - hm) * hi;
                }
                add_totals(a, base, slot, len, w, pl.vec);
            }
        }
        u += c1 - c0;
        if (u >= u1) return;  // the only piece, or the share's last
        __syncthreads();      // wave_m, wave_l and pool are free
        if (++vh == vheads) {
            vh = 0;
            row_at += row_chunks;
            do {
                ++row;
                len = __builtin_amdgcn_readfirstlane(kv_len(a.lens, row, a.max_len));
            } while (len == 0);
            row_chunks = chunks_of(len);
        }
        c0 = 0;
        c1 = min(row_chunks, u1 - u);
        part = 2 * blockIdx.x + 1;
    }
}

constexpr int JOIN_THREADS = ATTEND_THREADS;
constexpr int FEW_PARTS = 6;

// The second launch.  The first `sharers` workgroups add the weights to the
// totals, each for an equal share of the units of (row, head, chunk); the rows *
// q_heads after them join one query head's parts each.
template <int DIM>
__global__ __launch_bounds__(JOIN_THREADS) void kv_join_kernel(KvCache c, KvAttend a, AttendPlan pl) {
    constexpr int LANES = DIM / 4, SLICES = JOIN_THREADS / LANES;
    __shared__ __align__(16) float slice_o[SLICES][DIM];
    __shared__ float slice_l[SLICES];
    __shared__ float head_m[256], head_inv[256];
    const int tid = threadIdx.x, vheads = c.heads * pl.blocks;

    if ((int)blockIdx.x >= pl.sharers) {
        const int which = blockIdx.x - pl.sharers, row = which / a.q_heads, qh = which % a.q_heads;
        const int head = qh / pl.group, block = qh % pl.group / pl.block_heads, h = qh % pl.group % pl.block_heads;
        const int at = pl.before[row], chunks = pl.before[row + 1] - at;
        if (chunks == 0) return;
        const Parts parts = parts_of(c, pl, row, head * pl.blocks + block, at, chunks);
        if (parts.n == 1) return;  // written already
        const int d = tid % LANES * 4, slice = tid / LANES;
        float m = NEG_INF, l = 0.f;
        f32x4_kv o = {0.f, 0.f, 0.f, 0.f};
        for (int i = slice; i < parts.n; i += SLICES) {
            const int part = parts.place(i);
            const float pm = pl.part_ml[(part * 16 + h) * 2], ps = pl.part_ml[(part * 16 + h) * 2 + 1];
            const f32x4_kv x = *reinterpret_cast<const f32x4_kv *>(pl.part_o + ((int64_t)part * pl.block_heads + h) * DIM + d);
            const float top = fmaxf(m, pm);
            const float f0 = m == top ? 1.f : exp2f(m - top), f1 = pm == top ? 1.f : exp2f(pm - top);
            l = l * f0 + ps * f1;
            o = o * f0 + x * f1;
            m = top;
        }
        if (tid % LANES == 0) {
            head_m[slice] = m;
        }
        __syncthreads();
        float top = NEG_INF;
        for (int s = 0; s < SLICES; ++s) top = fmaxf(top, head_m[s]);
        const float f = m == top ? 1.f : exp2f(m - top);
        if (tid % LANES == 0) slice_l[slice] = l * f;
        *reinterpret_cast<f32x4_kv *>(&slice_o[slice][d]) = o * f;
        __syncthreads();
        if (tid < LANES) {
            float total = 0.f;
            f32x4_kv x = {0.f, 0.f, 0.f, 0.f};
            for (int s = 0; s < SLICES; ++s) {
                total += slice_l[s];
                x += *reinterpret_cast<f32x4_kv *>(&slice_o[s][d]);
            }
            const float inv = total == 0.f ? 0.f : (c.fp8 ? c.v_scale[head] : 1.f) / total;
            if (total == 0.f) x = f32x4_kv{0.f, 0.f, 0.f, 0.f};
            uint16_t *dst = a.out + (int64_t)row * a.out_ld + (int64_t)qh * DIM + d;
            *reinterpret_cast<u32x2_kv *>(dst) = u32x2_kv{pack_bf16(x[0] * inv, x[1] * inv), pack_bf16(x[2] * inv, x[3] * inv)};
        }
        return;
    }

    const int64_t all = (int64_t)pl.before[c.rows] * c.heads;
    const int64_t t0 = all * blockIdx.x / pl.sharers, t1 = all * (blockIdx.x + 1) / pl.sharers;
    if (t0 >= t1) return;
    int row = 0;
    for (int r0 = 0; r0 < c.rows; r0 += JOIN_THREADS) {
        const int r = r0 + tid;
        row += __syncthreads_count(r < c.rows && (int64_t)pl.before[r + 1] * c.heads <= t0);
    }
    for (int64_t t = t0; t < t1;) {
        const int at = pl.before[row], chunks = pl.before[row + 1] - at;
        if (chunks == 0) {
            ++row;
            continue;
        }
        const int64_t row0 = (int64_t)at * c.heads;
        const int head = (int)((t - row0) / chunks), c0 = (int)((t - row0) % chunks);
        const int c1 = (int)min((int64_t)chunks, c0 + (t1 - t));
        const int n = kv_len(a.lens, row, a.max_len);
        if (pl.blocks == 1 && chunks <= most_held(pl.block_heads) && parts_of(c, pl, row, head, at, chunks).n == 1) {
            t += c1 - c0;  // its workgroup did it
            if (head == c.heads - 1 && c1 == chunks) ++row;
            continue;
        }
        __syncthreads();
        // Each query head's m and 1 / sum over all of its parts: a thread for a head where
        // there are few parts, else a wave.  (4 rows of up to 4000 slots, 16 parts and
        // more: 23 us with waves, 35 with threads.)
        const Parts some = parts_of(c, pl, row, head * pl.blocks, at, chunks);
        const bool few = some.n <= FEW_PARTS;
        const int lane = tid & 63, width = few ? 1 : 64;
        for (int g = few ? tid : tid >> 6; g < pl.group; g += JOIN_THREADS / width) {
            const int block = g / pl.block_heads, h = g % pl.block_heads;
            const Parts parts = block ? parts_of(c, pl, row, head * pl.blocks + block, at, chunks) : some;
            const float *one = pl.whole + (((int64_t)row * vheads + head * pl.blocks + block) * 16 + h) * 2;
            float m = NEG_INF, l = 0.f;
            auto take = [&](int i) {
                const float *p = parts.n == 1 ? one : pl.part_ml + (parts.place(i) * 16 + h) * 2;
                const float pm = p[0], ps = p[1], top = fmaxf(m, pm);
                l = l * (m == top ? 1.f : exp2f(m - top)) + ps * (pm == top ? 1.f : exp2f(pm - top));
                m = top;
            };
            float top;
            if (few) {
                for (int i = 0; i < parts.n; ++i) take(i);
                top = m;
            } else {
                for (int i = lane; i < parts.n; i += 64) take(i);
                top = m;
#pragma unroll
                for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
                l *= m == top ? 1.f : exp2f(m - top);
#pragma unroll
                for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d);
            }
            if (few || lane == 0) {
                head_m[g] = top == NEG_INF ? 0.f : top;
                head_inv[g] = l == 0.f ? 0.f : weights_by(n) / l;
            }
        }
        __syncthreads();
        // Four slots of a thread, 32 threads of a unit.
        const int64_t base = ((int64_t)row * c.heads + head) * c.cap;
        for (int i = tid; i < (c1 - c0) * (CHUNK / 4); i += JOIN_THREADS) {
            const int chunk = c0 + i / (CHUNK / 4), in = i % (CHUNK / 4), slot = chunk * CHUNK + in * 4;
            if (slot >= n) continue;
            f32x4_kv w = {0.f, 0.f, 0.f, 0.f};
            for (int b = 0; b < pl.blocks; ++b) {
                const int heads = min(pl.block_heads, pl.group - b * pl.block_heads);
                const int64_t unit = (int64_t)at * vheads + (int64_t)(head * pl.blocks + b) * chunks + chunk;
                const float *s = pl.scores + (unit * (CHUNK / 4) + in) * 4 * pl.block_heads;
                const float *hm = head_m + b * pl.block_heads, *hi = head_inv + b * pl.block_heads;
                for (int h0 = 0; h0 < heads; h0 += 4) {  // four heads' scores in flight
                    f32x4_kv x[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h) x[h] = *reinterpret_cast<const f32x4_kv *>(s + min(h0 + h, heads - 1) * 4);
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        if (h0 + h < heads)
#pragma unroll
                            for (int e = 0; e < 4; ++e) w[e] += __builtin_amdgcn_exp2f(x[h][e] - hm[h0 + h]) * hi[h0 + h];
                }
            }
            add_totals(a, base, slot, n, w, pl.vec);
        }
        t += c1 - c0;
        if (head == c.heads - 1 && c1 == chunks) ++row;
    }
}

// The plan, its scratch laid out from `base`; returns the bytes (-1: more units than an int
// counts, or more workgroups than a launch takes).
static int64_t attend_plan(const KvCache &c, int q_heads, int max_len, bool weights, int cu_count, uint8_t *base,
                           AttendPlan *pl) {
    pl->group = q_heads / c.heads;
    pl->blocks = (pl->group + 15) / 16;
    pl->block_heads = (pl->group + pl->blocks - 1) / pl->blocks;
    const int64_t vheads = (int64_t)c.heads * pl->blocks, chunks = (max_len + CHUNK - 1) / CHUNK;
    const int64_t most = c.rows * vheads * chunks;
    if (most > INT32_MAX) return -1;
    // As many workgroups as run at once: two on a CU, one at 256 dims (registers).
    pl->wgs = (int)std::max<int64_t>(1, std::min<int64_t>(most, (int64_t)cu_count * (c.dim > 128 ? 1 : 2)));
    // One workgroup for each (row, head), undivided, where rows are short: up to four
    // units, whose steps 2 to 4 take about as long as the second launch that joins
    // parts; and up to about eight for each time that the workgroups fill the device,
    // when the last ones to run are a small share of all.  (96 rows of up to 600 slots,
    // 8 heads: 30 us so, 49 us in equal shares.)  With totals the scores of a row have
    // to stay in LDS, and the second launch, which then adds them up, is worth 12 steps.
    pl->undivided = chunks <= (weights ? 12 : 4) || (c.rows * vheads >= pl->wgs && chunks <= 8 * c.rows * vheads / pl->wgs);
    if (weights && (pl->blocks > 1 || chunks > most_held(pl->block_heads))) pl->undivided = 0;
    if (pl->undivided) pl->wgs = (int)(c.rows * vheads);
    // Totals: eight units for each step of a workgroup, and a few workgroups for each CU.
    pl->sharers = weights ? (int)std::max<int64_t>(1, std::min<int64_t>((most + 7) / 8, (int64_t)cu_count * 4)) : 0;
    if (!fits_launch(pl->undivided ? c.rows * vheads : (int64_t)c.rows * q_heads + pl->sharers, ATTEND_THREADS)) return -1;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        uint8_t *p = base ? base + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    pl->before = nullptr;
    pl->whole = pl->part_ml = pl->part_o = pl->scores = nullptr;
    pl->pieces = nullptr;
    if (pl->undivided) return 0;
    pl->before = (int32_t *)take((c.rows + 1) * 4);
    pl->pieces = (int32_t *)take((c.rows + 2) * 4);
    pl->part_ml = (float *)take((int64_t)pl->wgs * 2 * 16 * 2 * 4);
    pl->part_o = (float *)take((int64_t)pl->wgs * 2 * pl->block_heads * c.dim * 4);
    if (weights) {
        pl->whole = (float *)take(c.rows * vheads * 16 * 2 * 4);
        pl->scores = (float *)take(most * pl->block_heads * CHUNK * 4);
    }
    return at;
}

int64_t kv_attend_workspace_bytes(const KvCache &c, int q_heads, int max_len, bool weights, int cu_count) {
    AttendPlan pl;
    return attend_plan(c, q_heads, max_len, weights, cu_count, nullptr, &pl);
}

template <int DIM, bool FP8, bool PACK, bool SMALL>
static void launch_attend(const KvCache &c, const KvAttend &a, const AttendPlan &pl, bool once, hipStream_t stream) {
    const dim3 grid(pl.wgs), threads(ATTEND_THREADS);
    if (once && a.acc) hipLaunchKernelGGL((kv_attend_kernel<DIM, FP8, PACK, SMALL, true, true>), grid, threads, 0, stream, c, a, pl);
    else if (once) hipLaunchKernelGGL((kv_attend_kernel<DIM, FP8, PACK, SMALL, true, false>), grid, threads, 0, stream, c, a, pl);
    else if (a.acc) hipLaunchKernelGGL((kv_attend_kernel<DIM, FP8, PACK, SMALL, false, true>), grid, threads, 0, stream, c, a, pl);
    else hipLaunchKernelGGL((kv_attend_kernel<DIM, FP8, PACK, SMALL, false, false>), grid, threads, 0, stream, c, a, pl);
    if (!pl.undivided)
        hipLaunchKernelGGL((kv_join_kernel<DIM>), dim3((unsigned)(c.rows * a.q_heads + pl.sharers)), dim3(JOIN_THREADS), 0,
                           stream, c, a, pl);
}

template <int DIM, bool FP8>
static void launch_attend(const KvCache &c, const KvAttend &a, const AttendPlan &pl, hipStream_t stream) {
    // Loads that say their data is used once, if the rows may be too long for the
    // last-level cache (256 MB) to hold them until the next call: 537 MB take 90 us
    // with them and 102 without; 44 MB, called again, 22 and 21.
    const bool once = (int64_t)c.rows * c.heads * a.max_len * c.dim * (c.fp8 ? 2 : 4) > ((int64_t)256 << 20);
    const bool pack = pl.block_heads <= 8, small = c.page_log2 < 4;
    if (pack && small) launch_attend<DIM, FP8, true, true>(c, a, pl, once, stream);
    else if (pack) launch_attend<DIM, FP8, true, false>(c, a, pl, once, stream);
    else if (small) launch_attend<DIM, FP8, false, true>(c, a, pl, once, stream);
    else launch_attend<DIM, FP8, false, false>(c, a, pl, once, stream);
}

hipError_t launch_kv_attend(const KvCache &c, const KvAttend &a, int cu_count, hipStream_t stream) {
    AttendPlan pl;
    attend_plan(c, a.q_heads, a.max_len, a.acc != nullptr, cu_count, a.ws, &pl);
    pl.vec = c.cap % 4 == 0 && (((uintptr_t)a.acc | (uintptr_t)a.acc_out) & 15) == 0;
    switch (c.dim) {
    case 64:
        if (c.fp8) launch_attend<64, true>(c, a, pl, stream); else launch_attend<64, false>(c, a, pl, stream);
        break;
    case 128:
        if (c.fp8) launch_attend<128, true>(c, a, pl, stream); else launch_attend<128, false>(c, a, pl, stream);
        break;
    default:
        if (c.fp8) launch_attend<256, true>(c, a, pl, stream); else launch_attend<256, false>(c, a, pl, stream);
        break;
    }
    return hipGetLastError();
}

}  // namespace nbw
