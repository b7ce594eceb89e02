// kv_shared.hip -- attention of each row's new tokens over its cached slots, where
// groups of rows share a prefix that is read once for all of them, gfx950.
//
// For a line, a query head of a new token, with the n slots that the token sees
//     s_j = scale q.k_j,   o = sum_j 2^(s_j' - m) v_j / sum_j 2^(s_j' - m),
// s' = s log2(e), with any m near the largest s'.  Slots are cut in segments: a group's
// prefix, with all lines of the group, and each row's own slots behind it, with the row's
// lines.  What a segment gives a line, (m, sum, o), is joined in a last launch.
//
// Four launches: the segments' sizes; the prefixes; the rows' own slots; the join.  In the
// middle two a workgroup takes a block of 32 LW lines of one head over a run of slots, its
// SW waves along the slots sharing each tile of them: many lines (LW = 4, SW = 1) read
// each key and value from LDS for 32 lines each, few lines (LW = 1, SW = 4) are bound by
// the cache's bytes, of which each wave takes its own 32 slots.  The units of all segments, 128
// slots of a block, are divided in equal shares over as many workgroups as run at once,
// whatever the lengths.
//
// A tile goes from memory through registers, asked for a tile ahead, to LDS (8-bit
// values widened to bf16 on the way), in 16-byte pieces whose place within a row is turned by the
// row's number so that no two lanes of a half wave meet in a bank.  Then on
// v_mfma_f32_32x32x16_bf16, with a line in each lane throughout:
//  - S^T = K Q^T: lane l has line l % 32 and of 32 slots the ones 8 (i / 4) + 4 (l / 32) + i % 4
//    in its registers i = 0..15, so the maximum and the sum need one exchange, between the halves;
//  - O^T = V^T P^T: these are the slots of P^T that the lane has to supply, if the product's inner
//    index 8 (l / 32) + j of step u stands for register 8 u + j; V^T comes from LDS by
//    transposing loads of four slots each, and o has its line in the lane too: rescaling it
//    is a product with the lane's own number.
//
// The weights are rounded to bf16, half a step of 2^-8, for the second product; 24 bits, as
// in the attention of one token, would take three times its matrix instructions, and the prefix
// is bound by them.  The sum is taken over the rounded ones, so that an average of equal
// values is exact and the error is that of the weights' differences.
//
// The running maximum m of a line is only raised, and o and the sum rescaled, when a score
// passes it by more than 8 (a factor of 2^8).
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
    int chunks, blocks;  // units of a head: of a block of lines, and blocks
    int pad;
};

// The call's division of work and its scratch.
struct SharedPlan {
    int group;                   // query heads of a head
    int wgs;                     // workgroups of the launch that attends
    int2 *tokens;                // [tokens] the token's row, or -1, and that row's group, or -1
    int32_t *sees;               // [tokens] slots that it sees
    int32_t *shares;             // [2] of the workgroups, those of each side
    struct Side {                // 0: the groups' prefixes, 1: the rows' own slots
        int lines, segments;     // lines of a block
        Segment *segment;        // [segments]
        int64_t *units;          // [segments + 1] units before each segment
        float *first_ml, *first_o;  // [tokens][q_heads][2], [..][dim]: a line's part from its segment's first slot on
        float *more_ml, *more_o;    // [wgs][lines][2], [..][dim]: the part that a workgroup begins elsewhere
    } side[2];
};

__device__ __forceinline__ int bounded(int x, int low, int high) { return min(max(x, low), high); }
__device__ __forceinline__ int first_token(const KvAttendShared &a, int row) {
    return a.cu ? bounded(a.cu[row], 0, a.tokens) : row;
}

// The number of entries 1 .. n of an ascending array that are at most x.
__device__ __forceinline__ int ended_by(const int32_t *ends, int n, int x) {
    int low = 0, high = n;
    while (low < high) {
        const int mid = (low + high) / 2;
        if (ends[mid + 1] <= x) low = mid + 1;
        else high = mid;
    }
    return low;
}
__device__ __forceinline__ int group_of(const KvAttendShared &a, int row) {
    if (!a.group_rows) return -1;
    const int g = ended_by(a.group_rows, a.groups, row);
    return g < a.groups && a.group_rows[g] <= row ? g : -1;
}

// The last workgroup of the launch counts the segments' units, the others find each token's row.
constexpr int PLAN_THREADS = 256;
__global__ __launch_bounds__(PLAN_THREADS) void kv_shared_plan_kernel(KvCache c, KvAttendShared a, SharedPlan pl) {
    __shared__ int64_t s_wave[PLAN_THREADS / 64], s_all[2];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (blockIdx.x + 1 < gridDim.x) {
        const int token = blockIdx.x * PLAN_THREADS + tid;
        if (token >= a.tokens) return;
        int row = token, behind = 0;
        if (a.cu) {
            row = ended_by(a.cu, c.rows, token);
            if (row < c.rows && a.cu[row] <= token) behind = min(a.cu[row + 1], a.tokens) - 1 - token;
            else row = -1;
        }
        pl.tokens[token] = int2{row, row < 0 ? -1 : group_of(a, row)};
        pl.sees[token] = row < 0 ? 0 : max(kv_len(a.lens, row, a.max_len) - behind, 0);
        return;
    }
    // Running sums of the segments' units, a strip of segments for each thread.
    for (int which = 0; which < 2; ++which) {
        const auto &side = pl.side[which];
        const int n = side.segments;
        const int strip = (n + PLAN_THREADS - 1) / PLAN_THREADS, s0 = min(tid * strip, n), s1 = min(s0 + strip, n);
        int64_t mine = 0;
        for (int s = s0; s < s1; ++s) {
            Segment x = {s, 0, 0, 0, 0, 0, 0, 0};
            if (which) {
                const int g = group_of(a, s), t1 = first_token(a, s + 1);
                x.token = first_token(a, s);
                x.tokens = max(t1 - x.token, 0);
                x.start = g < 0 ? 0 : bounded(a.prefix[g], 0, a.max_len);
                x.end = kv_len(a.lens, s, a.max_len);
            } else {
                const int r0 = bounded(a.group_rows[s], 0, c.rows), r1 = bounded(a.group_rows[s + 1], 0, c.rows);
                x.row = r0;
                x.token = first_token(a, r0);
                x.tokens = r0 < r1 ? max(first_token(a, r1) - x.token, 0) : 0;
                x.end = bounded(a.prefix[s], 0, a.max_len);
            }
            x.chunks = x.tokens > 0 && x.end > x.start ? (x.end - x.start + UNIT - 1) / UNIT : 0;
            x.blocks = (int)(((int64_t)x.tokens * pl.group + side.lines - 1) / side.lines);
            side.segment[s] = x;
            mine += (int64_t)c.heads * x.blocks * x.chunks;
        }
        int64_t upto = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t x = __shfl_up(upto, d);
            if (lane >= d) upto += x;
        }
        if (lane == 63) s_wave[wave] = upto;
        __syncthreads();
        for (int w = 0; w < wave; ++w) upto += s_wave[w];
        int64_t at = upto - mine;
        for (int s = s0; s < s1; ++s) {
            side.units[s] = at;
            at += (int64_t)c.heads * side.segment[s].blocks * side.segment[s].chunks;
        }
        if (tid == PLAN_THREADS - 1) side.units[n] = s_all[which] = upto;
        __syncthreads();
    }
    if (tid == 0) {
        // Workgroups by the sides' units, one for each unit at the most and one for a side that has any.
        const int64_t u0 = s_all[0], u1 = s_all[1];
        int64_t n0 = u0, n1 = u1;
        if (u0 + u1 > pl.wgs) {
            n0 = (pl.wgs * u0 + (u0 + u1) / 2) / (u0 + u1);
            n0 = min(max(n0, (int64_t)(u0 > 0)), (int64_t)pl.wgs - (u1 > 0));
            n1 = min(pl.wgs - n0, u1);
        }
        pl.shares[0] = (int)n0;
        pl.shares[1] = (int)n1;
    }
}

// The workgroup whose share a unit is in.
__device__ __forceinline__ int owner_of(int64_t unit, int64_t units, int shares) {
    return (int)(((unit + 1) * shares - 1) / units);
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

// How a workgroup takes its lines.  Few: 32, and of each 128 slots a wave has 32, in LDS of its
// own, so that no wave waits for another.  Many: 128, 32 to a wave, over tiles in two buffers
// that the waves fill together.
template <int DIM, bool FEW>
struct Shape {
    static constexpr int LINES = FEW ? 32 : 32 * SHARED_WAVES;
    static constexpr int SUBS = !FEW && DIM < 256 ? 2 : 1;       // runs of 32 slots that a wave takes at once
    static constexpr int TILE = 32 * SUBS;                       // slots in LDS, of a wave, or of all
    static constexpr int STEP = FEW ? TILE * SHARED_WAVES : TILE; // slots from one of a wave's tiles to the next
    static constexpr int PIECES = DIM / 8;                       // of a slot's row, 16 bytes each
    static constexpr int ROWS = 64 / PIECES;                     // that a wave's lanes have a piece each of
    static constexpr int FILLED = FEW ? TILE : TILE / SHARED_WAVES; // rows of a tile that a wave fills
    static constexpr int LOADS = FILLED / ROWS;                  // of a lane for them, of keys and of values
    static constexpr int ROW = DIM * 2;
    static constexpr int PART = 32 * (DIM + 4) * 4;              // a wave's o, its rows 16 bytes past the banks' turn
    static constexpr int OWN = std::max(2 * TILE * ROW, PART);   // of a wave
    static constexpr int BYTES = FEW ? OWN * SHARED_WAVES : 4 * TILE * ROW;
};

// 16 bytes of each lane to LDS, side by side from `lds` on, which is the same for all of them.  Written out, as the
// compiler puts a wait for all such loads before each transposing read, whatever that reads; what
// has to have arrived is said by wait_loads.  No register is written.
__device__ __forceinline__ void load_to_lds(const uint8_t *p, uint8_t *lds) {
    const uint32_t at = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(__attribute__((address_space(3))) void *)lds);
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "s"(at) : "memory", "m0");
}

struct SharedLds {
    uint8_t *pool;
    int (*bad)[SHARED_WAVES];   // by buffer and wave: a page of the tile is not there
    float (*m)[32], (*l)[32];   // by wave and line
};

// One workgroup's share of a side's units.
template <int DIM, bool FP8, bool FEW>
__device__ __forceinline__ void attend_share(const KvCache &c, const KvAttendShared &a, const SharedPlan &pl, int which, int share,
                                             int shares, const SharedLds &lds) {
    using X = Shape<DIM, FEW>;
    constexpr int TILE = X::TILE, SUBS = X::SUBS, PIECES = X::PIECES, LOADS = X::LOADS, ROW = X::ROW;
    constexpr int R = 256 / DIM;  // rows of a tile in 512 bytes, one turn of the banks
    constexpr int DB = DIM / 32, QF = DIM / 16;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = lane >> 5, col = lane & 31;
    const auto &side = pl.side[which];
    const int64_t units = side.units[side.segments];
    int64_t u = units * share / shares;
    const int64_t u1 = units * (share + 1) / shares;
    int seg = 0;  // segments that end at or before u
    for (int at = 0; at < side.segments; at += 64) {
        const int n = __popcll(__ballot(at + lane < side.segments && side.units[at + lane + 1] <= u));
        seg += n;
        if (n < 64) break;
    }

    // A row of a tile has its pieces at places turned by the row's number s: by (s / R) % PIECES for
    // keys, whose readers have 32 rows side by side; by 4 ((s / R) % (8 / R)) for values, whose readers
    // have 8 rows and 4 pieces.  A lane fills place l % PIECES of rows ROWS i + l / PIECES, of which s / R is
    // 2 i + l / 32 (from a multiple of 8 on), so the piece it loads for i differs from that for 0 by bits of i.
    const int first_row = FEW ? 0 : wave * X::FILLED;  // that the wave fills
    const int fill_row = lane / PIECES;
    const int k_fill = ((lane % PIECES) ^ ((first_row / R + half) & (PIECES - 1))) << 4, v_fill = ((lane % PIECES) ^ (half << 2)) << 4;
    const int k_read = col * ROW, k_turn = (half ^ ((col / R) & (PIECES - 1))) << 4;
    const int v_slot = 4 * half + (lane & 15) / 4;
    const int v_turn = ((v_slot / R) & (8 / R - 1)) << 6;
    const int v_read = v_slot * ROW + (2 * ((lane >> 4) & 1) + (lane & 3) / 2) * 16 + (lane & 1) * 8;
    uint8_t *const own = lds.pool + (FEW ? wave * X::OWN : 0);

    for (;;) {  // a piece: chunks [c0, c1) of one block of a segment's lines
        const Segment sg = side.segment[seg];
        const int64_t in = u - side.units[seg];
        const int per_head = sg.blocks * sg.chunks, head = (int)(in / per_head), rest = (int)(in % per_head);
        const int block = rest / sg.chunks, c0 = rest % sg.chunks, c1 = (int)min((int64_t)sg.chunks, c0 + (u1 - u));
        const int nlines = min(X::LINES, sg.tokens * pl.group - block * X::LINES);
        const int from = sg.start + c0 * UNIT + (FEW ? wave * TILE : 0);  // the wave's first slot
        const int32_t *table = c.table + (int64_t)sg.row * c.table_ld;

        // The page of a slot of a tile that the wave fills: lane l has that of its row l % FILLED.
        int32_t page;
        auto ask_page = [&](int tile) {
            page = table[min(from + tile * X::STEP + first_row + lane % X::FILLED, c.cap - 1) >> c.page_log2];
        };
        ask_page(0);

        const int line = FEW ? col : wave * 32 + col;
        const bool valid = line < nlines;
        const int seg_line = block * X::LINES + (valid ? line : 0);
        const int token = sg.token + seg_line / pl.group, q_head = head * pl.group + seg_line % pl.group;
        u32x4_kv q[QF];
        {
            const uint16_t *src = a.q + (int64_t)token * a.q_ld + (int64_t)q_head * DIM + half * 8;
            const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
            for (int f = 0; f < QF; ++f) {
                q[f] = *reinterpret_cast<const u32x4_kv *>(src + f * 16);
#pragma unroll
                for (int e = 0; e < 4; ++e) q[f][e] = valid ? q[f][e] ^ flip : 0u;
            }
        }
        // The last slot that any line sees: a row's later tokens see more.
        const int end = which ? min(sg.end, pl.sees[sg.token + (block * X::LINES + nlines - 1) / pl.group]) : sg.end;
        const int to = min(sg.start + c1 * UNIT, end);
        const int tiles = to > from ? (to - from + X::STEP - 1) / X::STEP : 0;
        const int sees = valid ? min(pl.sees[token], to) : INT32_MAX;
        const int least = -wave_max(-sees), most = wave_max(valid ? sees : 0);
        const float by = fabsf(a.scale) * 1.44269504088896340736f * (FP8 ? c.k_scale[head] : 1.f);
        // Weights are up to 2^RAISE, and as many meet the values as the segment has slots: times a
        // power of two, in their exponent, they sum to 1 at the most, and finite values cannot run over.
        const int n = sg.end - sg.start;
        const float room = RAISE + (n > 1 ? 32 - __builtin_clz(n - 1) : 0);

        // A tile's rows of a pool, by numbers: a table of one word for each of the wave's rows, in its lanes.
        uint32_t rows = 0;
        auto find = [&](int tile) {  // the page asked for last is the tile's
            const int slot = from + tile * X::STEP + first_row + lane % X::FILLED;
            const bool there = page >= 0 && page < c.pages;
            rows = (((uint32_t)(there ? page : 0) * (uint32_t)c.heads + (uint32_t)head) << c.page_log2) +
                   (uint32_t)(slot & ((1 << c.page_log2) - 1));
            return __any(!there);
        };
        // 8-bit values come through registers, to be widened.
        u32x2_kv raw[FP8 ? 2 : 1][LOADS];
        auto load = [&](bool values, uint8_t *to_lds) {
            int fill = values ? v_fill : k_fill, row = fill_row;
            again(fill, row);
            const uint8_t *pool = values ? c.v : c.k;
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const uint32_t r = __shfl(rows, row + i * X::ROWS);
                const int at = values ? fill ^ (((2 * i) & (8 / R - 1)) << 6) : fill ^ (2 * i << 4);
                if constexpr (FP8) {
                    raw[values][i] = *reinterpret_cast<const u32x2_kv *>(pool + (int64_t)r * DIM + (at >> 1));
                } else {
                    load_to_lds(pool + (int64_t)r * ROW + at, to_lds + i * 1024);
                }
            }
        };
        auto widen = [&](bool values, uint8_t *to_lds) {
            if constexpr (FP8) {
#pragma unroll
                for (int i = 0; i < LOADS; ++i) {
                    const u32x2_kv w = raw[values][i];
                    *reinterpret_cast<u32x4_kv *>(to_lds + i * 1024 + lane * 16) =
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
        u32x4_kv p[SUBS][2];

        // S^T of the tile whose keys are at kb.
        auto scores = [&](const uint8_t *kb) {
            int row = k_read, way = k_turn;
            again(row, way);
#pragma unroll
            for (int b = 0; b < SUBS; ++b) {
#pragma unroll
                for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
#pragma unroll
                for (int f = 0; f < QF; ++f) {
                    const u32x4_kv kf = *reinterpret_cast<const u32x4_kv *>(kb + b * 32 * ROW + row + (way ^ (f << 5)));
                    s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_sh, kf),
                                                                   __builtin_bit_cast(bf16x8_sh, q[f]), s[b], 0, 0, 0);
                }
            }
        };
        // The weights, in s and rounded in p; `first` is the tile's first slot, `all` says that every line sees the whole tile.
        auto weigh = [&](int first, auto all, const uint32_t *there) {
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
                for (int i = 0; i < 16; ++i) top = fmaxf(top, s[b][i]);
            top *= by;  // by is positive: the largest stays the largest
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
            const float ref = m == NEG_INF ? 0.f : m;
            float part = 0.f;  // of a long sum, so that few roundings follow each other
#pragma unroll
            for (int b = 0; b < SUBS; ++b)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[b][2 * i] = __builtin_amdgcn_exp2f(fmaf(s[b][2 * i], by, -ref));
                    s[b][2 * i + 1] = __builtin_amdgcn_exp2f(fmaf(s[b][2 * i + 1], by, -ref));
                    const bf16x2_sh two = {(__bf16)s[b][2 * i], (__bf16)s[b][2 * i + 1]};
                    part = __builtin_amdgcn_fdot2_f32_bf16(two, bf16x2_sh{(__bf16)1.f, (__bf16)1.f}, part, false);
                    p[b][i / 4][i % 4] = __builtin_bit_cast(uint32_t, two);
                }
            sum += part;
        };
        // O^T with the values at vb.
        auto add = [&](const uint8_t *vb, auto finite) {
            int row = v_read, way = v_turn;
            again(row, way);
#pragma unroll
            for (int b = 0; b < SUBS; ++b)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const uint8_t *src = vb + (b * 32 + 16 * k) * ROW + row + ((d << 6) ^ way);
                        const u32x2_kv v0 = transposed(src), v1 = transposed(src + 8 * ROW);
                        u32x4_kv vf = {v0[0], v0[1], v1[0], v1[1]};
                        if constexpr (decltype(finite)::value) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if ((vf[e] & 0x7F80u) == 0x7F80u) vf[e] &= 0xFFFF0000u;
                                if ((vf[e] & 0x7F800000u) == 0x7F800000u) vf[e] &= 0x0000FFFFu;
                            }
                        }
                        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_sh, vf),
                                                                       __builtin_bit_cast(bf16x8_sh, p[b][k]), o[d], 0, 0, 0);
                    }
        };
        // The same where a slot may not count, for a line or for all: its weight is 0, but what
        // lies there may be NaN or infinite.  Such values are left out of the product and added to the
        // lines that do see them, one slot after the other.
        auto add_with_care = [&](const uint8_t *vb, int first, const uint32_t *there) {
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
                add(vb, std::false_type());
                return;
            }
            add(vb, std::true_type());
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
                    const int row = b * 32 + j, turn = ((row / R) & (8 / R - 1)) << 6;
                    const uint8_t *src = vb + row * ROW + dim0 * 2;
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        __builtin_amdgcn_sched_barrier(0);  // few loads at a time
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
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
            uint8_t *kb = own, *vb = own + TILE * ROW;
            bool missing = false;
            if (tiles > 0) {
                missing = find(0);
                load(false, kb);
                load(true, vb);
                ask_page(min(1, tiles - 1));
            }
            auto step = [&](int t, auto all) {
                const int first = from + t * X::STEP;
                if constexpr (FP8) widen(false, kb);
                else wait_loads<LOADS + 1>();  // the values and a page number
                scores(kb);
                wait_lds();
                if constexpr (!FP8) wait_loads<0>();
                uint32_t there[SUBS];
                if constexpr (!decltype(all)::value) present(first, missing, there);
                missing = find(min(t + 1, tiles - 1));
                if constexpr (FP8) widen(true, vb);
                load(false, kb);
                weigh(first, all, there);
                if constexpr (decltype(all)::value) add(vb, std::false_type());
                else add_with_care(vb, first, there);
                wait_lds();
                load(true, vb);
                ask_page(min(t + 2, tiles - 1));
            };
            int t = 0;
            for (; t < tiles && from + t * X::STEP + TILE <= least && !missing; ++t) step(t, std::true_type());
            for (; t < tiles; ++t) step(t, std::false_type());
            if constexpr (!FP8) wait_loads<0>();
        } else {
            auto buf = [&](int t) { return own + (t & 1) * 2 * TILE * ROW; };
            auto fill = [&](int t) {
                const bool any = find(t);
                if (lane == 0) lds.bad[t & 1][wave] = any;
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
            auto missing = [&](int t) {
                bool any = false;
#pragma unroll
                for (int w = 0; w < SHARED_WAVES; ++w) any = any || lds.bad[t & 1][w];
                return (bool)__builtin_amdgcn_readfirstlane(any);
            };
            if (tiles > 0) {
                fill(0);
                ask_page(min(1, tiles - 1));
                arrive(0);
            }
            // Each wave meets the others once a tile, whichever of the two loops it is in.
            auto step = [&](int t, auto all) {
                if (t + 1 < tiles) {
                    fill(t + 1);
                    ask_page(min(t + 2, tiles - 1));
                }
                const int first = from + t * X::STEP;
                const uint8_t *kb = buf(t), *vb = kb + TILE * ROW;
                if constexpr (decltype(all)::value) {
                    scores(kb);
                    weigh(first, all, nullptr);
                    add(vb, std::false_type());
                } else if (first < most) {
                    uint32_t there[SUBS];
                    present(first, missing(t), there);
                    scores(kb);
                    weigh(first, all, there);
                    add_with_care(vb, first, there);
                }
                if (t + 1 < tiles) arrive(t + 1);
            };
            int t = 0;
            for (; t < tiles && from + t * X::STEP + TILE <= least && !missing(t); ++t) step(t, std::true_type());
            for (; t < tiles; ++t) step(t, std::false_type());
        }

        // The piece's result.  One that has all that its lines see is the result; others wait for the join.
        sum += __shfl_xor(sum, 32);
        const bool sole = which && sg.start == 0 && c0 == 0 && c1 == sg.chunks;
        const float v_by = FP8 ? c.v_scale[head] : 1.f;
        auto store = [&](int ln, int d, f32x4_sh x, float mm, float total) {  // dims d..d+3 of a line of the block
            const int sl = block * X::LINES + ln;
            const int64_t t = sg.token + sl / pl.group, qh = head * pl.group + sl % pl.group;
            if (sole) {
                const float inv = total == 0.f ? 0.f : v_by / total;
                if (total == 0.f) x = f32x4_sh{0.f, 0.f, 0.f, 0.f};  // nothing to attend to, whatever the values are
                *reinterpret_cast<u32x2_kv *>(a.out + t * a.out_ld + qh * DIM + d) =
                    u32x2_kv{bf16_pair(x[0] * inv, x[1] * inv), bf16_pair(x[2] * inv, x[3] * inv)};
            } else {
                const int64_t at = c0 == 0 ? t * a.q_heads + qh : (int64_t)share * X::LINES + ln;
                float *ml = c0 == 0 ? side.first_ml : side.more_ml, *po = c0 == 0 ? side.first_o : side.more_o;
                *reinterpret_cast<f32x4_sh *>(po + at * DIM + d) = x;
                if (d == 0) {
                    ml[2 * at] = mm;
                    ml[2 * at + 1] = total;
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
        u += c1 - c0;
        if (u >= u1) return;
        meet();  // the pool and the sums are free
        while (side.units[seg + 1] <= u) ++seg;
    }
}

template <int DIM, bool FP8>
__global__ __launch_bounds__(SHARED_THREADS, DIM > 128 ? 1 : 2) void kv_shared_kernel(KvCache c, KvAttendShared a, SharedPlan pl) {
    __shared__ __align__(16) uint8_t pool[std::max(Shape<DIM, true>::BYTES, Shape<DIM, false>::BYTES)];
    __shared__ __align__(16) int s_bad[2][SHARED_WAVES];
    __shared__ float s_m[SHARED_WAVES][32], s_l[SHARED_WAVES][32];
    const SharedLds lds = {pool, s_bad, s_m, s_l};
    const int n0 = pl.shares[0], n1 = pl.shares[1], b = (int)blockIdx.x;
    if (b >= n0 + n1) return;
    const int which = b >= n0;
    // Workgroups go to the 8 XCDs in turn; neighbouring shares, which meet the same keys, go to one.
    int share = b - n0;
    if (!which) share = b % 8 * (n0 / 8) + min(b % 8, n0 % 8) + b / 8;
    if (pl.side[which].lines == Shape<DIM, true>::LINES) attend_share<DIM, FP8, true>(c, a, pl, which, share, which ? n1 : n0, lds);
    else attend_share<DIM, FP8, false>(c, a, pl, which, share, which ? n1 : n0, lds);
}

// The last launch: each line's parts, in a fixed order, by a wave.
constexpr int JOIN_THREADS = 256;
template <int DIM>
__global__ __launch_bounds__(JOIN_THREADS) void kv_shared_join_kernel(KvCache c, KvAttendShared a, SharedPlan pl) {
    constexpr int LANES = DIM / 4, SLICES = 64 / LANES;  // lanes of a part, four dims each, and parts taken side by side
    const int lane = threadIdx.x & 63, d = lane % LANES * 4;
    const int line = __builtin_amdgcn_readfirstlane((int)((int64_t)blockIdx.x * (JOIN_THREADS / 64) + (threadIdx.x >> 6)));
    if (line >= a.tokens * a.q_heads) return;
    const int token = line / a.q_heads, qh = line % a.q_heads, head = qh / pl.group;
    const int2 of = pl.tokens[token];
    if (of.x < 0) return;
    int first[2] = {0, 0}, n[2] = {0, 0}, in_block[2] = {0, 0};  // of each side: the first part's share, parts, line of its block
    bool written = false;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const int seg = which ? of.x : of.y;
        if (seg < 0) continue;
        const auto &side = pl.side[which];
        const Segment sg = side.segment[seg];
        if (sg.chunks == 0) continue;
        const int64_t units = side.units[side.segments];
        const int shares = pl.shares[which];
        const int in = (token - sg.token) * pl.group + qh % pl.group, block = in / side.lines;
        const int64_t at = side.units[seg] + ((int64_t)head * sg.blocks + block) * sg.chunks;
        first[which] = owner_of(at, units, shares);
        n[which] = owner_of(at + sg.chunks - 1, units, shares) - first[which] + 1;
        in_block[which] = in % side.lines;
        written = which && sg.start == 0 && n[1] == 1;
    }
    if (written) return;
    auto place = [&](int i, const float *&ml, const float *&po) {
        const int which = i >= n[0];
        const auto &side = pl.side[which];
        i -= which ? n[0] : 0;
        const int64_t at = i == 0 ? line : (int64_t)(first[which] + i) * side.lines + in_block[which];
        ml = (i == 0 ? side.first_ml : side.more_ml) + 2 * at;
        po = (i == 0 ? side.first_o : side.more_o) + at * DIM + d;
    };
    const int parts = n[0] + n[1];
    const float *ml, *po;
    // The largest m, and each part's share of the sum before any meets its o: finite values cannot run over.
    float top = NEG_INF, total = 0.f;
    for (int i = lane; i < parts; i += 64) {
        place(i, ml, po);
        const float m = ml[0], up = fmaxf(top, m);
        total = total * (top == up ? 1.f : __builtin_amdgcn_exp2f(top - up)) + ml[1] * (m == up ? 1.f : __builtin_amdgcn_exp2f(m - up));
        top = up;
    }
    float all = top;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) all = fmaxf(all, __shfl_xor(all, s));
    total *= top == all ? 1.f : __builtin_amdgcn_exp2f(top - all);
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) total += __shfl_xor(total, s);
    const float inv = total == 0.f ? 0.f : 1.f / total;
    f32x4_sh x = {0.f, 0.f, 0.f, 0.f};
    constexpr int AHEAD = 4;
    for (int i0 = 0; i0 < parts; i0 += AHEAD * SLICES) {
        f32x4_sh y[AHEAD];
        float m[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            place(min(i0 + k * SLICES + lane / LANES, parts - 1), ml, po);
            m[k] = ml[0];
            y[k] = *reinterpret_cast<const f32x4_sh *>(po);
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k)
            if (i0 + k * SLICES + lane / LANES < parts) x += y[k] * ((m[k] == all ? 1.f : __builtin_amdgcn_exp2f(m[k] - all)) * inv);
    }
#pragma unroll
    for (int s = LANES; s < 64; s <<= 1)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += __shfl_xor(x[e], s);
    if (total == 0.f) x = f32x4_sh{0.f, 0.f, 0.f, 0.f};  // nothing to attend to, whatever the values are
    if (c.fp8) x *= c.v_scale[head];
    if (lane < LANES)
        *reinterpret_cast<u32x2_kv *>(a.out + (int64_t)token * a.out_ld + (int64_t)qh * DIM + d) =
            u32x2_kv{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])};
}

// The plan, its scratch laid out from `base`; returns the bytes (-1: more than a launch takes).
static int64_t shared_plan(const KvCache &c, int q_heads, int tokens, int groups, int max_len, int cu_count, uint8_t *base,
                           SharedPlan *pl) {
    if ((c.pages * c.heads) >> (32 - c.page_log2)) return -1;  // a pool's rows are counted in 32 bits
    pl->group = q_heads / c.heads;
    const int64_t lines = (int64_t)tokens * pl->group, chunks = (max_len + UNIT - 1) / UNIT;
    int64_t units = 0;
    for (int which = 0; which < 2; ++which) {
        auto &side = pl->side[which];
        side.segments = which ? c.rows : groups;
        const int64_t mean = side.segments ? (lines + side.segments - 1) / side.segments : 0;  // lines of a segment
        side.lines = mean <= 32 ? 32 : 128;
        if (side.segments) units += (lines / side.lines + side.segments) * c.heads * chunks;
        if (units > INT32_MAX) return -1;
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
    pl->shares = (int32_t *)take(8);
    for (int which = 0; which < 2; ++which) {
        auto &side = pl->side[which];
        const int64_t all = side.segments ? (int64_t)tokens * q_heads : 0;
        const int64_t more = side.segments ? (int64_t)pl->wgs * side.lines : 0;
        side.segment = (Segment *)take((int64_t)side.segments * sizeof(Segment));
        side.units = (int64_t *)take(((int64_t)side.segments + 1) * 8);
        side.first_ml = (float *)take(all * 8);
        side.first_o = (float *)take(all * c.dim * 4);
        side.more_ml = (float *)take(more * 8);
        side.more_o = (float *)take(more * c.dim * 4);
    }
    return at;
}

int64_t kv_attend_shared_workspace_bytes(const KvCache &c, int q_heads, int tokens, int groups, int max_len, int cu_count) {
    SharedPlan pl;
    return shared_plan(c, q_heads, tokens, groups, max_len, cu_count, nullptr, &pl);
}

template <int DIM>
static void launch_shared(const KvCache &c, const KvAttendShared &a, const SharedPlan &pl, hipStream_t stream) {
    const dim3 grid((unsigned)pl.wgs), threads(SHARED_THREADS);
    if (c.fp8) hipLaunchKernelGGL((kv_shared_kernel<DIM, true>), grid, threads, 0, stream, c, a, pl);
    else hipLaunchKernelGGL((kv_shared_kernel<DIM, false>), grid, threads, 0, stream, c, a, pl);
    const int64_t lines = (int64_t)a.tokens * a.q_heads;
    constexpr int EACH = JOIN_THREADS / 64;
    hipLaunchKernelGGL((kv_shared_join_kernel<DIM>), dim3((unsigned)((lines + EACH - 1) / EACH)), dim3(JOIN_THREADS), 0, stream,
                       c, a, pl);
}

hipError_t launch_kv_attend_shared(const KvCache &c, const KvAttendShared &a, int cu_count, hipStream_t stream) {
    SharedPlan pl;
    shared_plan(c, a.q_heads, a.tokens, a.groups, a.max_len, cu_count, a.ws, &pl);
    const unsigned finders = (unsigned)((a.tokens + PLAN_THREADS - 1) / PLAN_THREADS);
    hipLaunchKernelGGL(kv_shared_plan_kernel, dim3(finders + 1), dim3(PLAN_THREADS), 0, stream, c, a, pl);
    switch (c.dim) {
    case 64: launch_shared<64>(c, a, pl, stream); break;
    case 128: launch_shared<128>(c, a, pl, stream); break;
    default: launch_shared<256>(c, a, pl, stream); break;
    }
    return hipGetLastError();
}

}  // namespace nbw
