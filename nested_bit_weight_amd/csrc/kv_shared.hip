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

constexpr int UNIT = 128;    // slots of a unit of work
constexpr float RAISE = 8.f; // how far a score may pass the running maximum

#define NEG_INF (-__builtin_inff())

// The call's division of work and its scratch.
struct SharedPlan {
    int group;                   // query heads of a head
    int32_t *token_row;          // [tokens] the token's row, or -1
    int32_t *token_sees;         // [tokens] slots that it sees
    int32_t *row_prefix;         // [rows] the row's slots within its group's prefix
    int32_t *row_group;          // [rows] the row's group, or -1
    struct Side {                // 0: the groups' prefixes, 1: the rows' own slots
        int wgs, lines;          // workgroups, and lines of a block
        int64_t *units;          // [segments + 1] units before each segment
        float *first_ml, *first_o;  // [tokens][q_heads][2], [..][dim]: a line's part from its segment's first slot on
        float *more_ml, *more_o;    // [wgs][lines][2], [..][dim]: the part that a workgroup begins elsewhere
    } side[2];
};

// Lines and slots of a segment.
struct Segment {
    int row;            // whose table holds its slots
    int token, tokens;  // its lines' tokens
    int start, end;     // its slots
};
__device__ __forceinline__ int bounded(int x, int low, int high) { return min(max(x, low), high); }
__device__ __forceinline__ int first_token(const KvAttendShared &a, int row) {
    return a.cu ? bounded(a.cu[row], 0, a.tokens) : row;
}
__device__ __forceinline__ Segment prefix_of(const KvCache &c, const KvAttendShared &a, int g) {
    const int r0 = bounded(a.group_rows[g], 0, c.rows), r1 = bounded(a.group_rows[g + 1], 0, c.rows);
    const int t0 = first_token(a, r0), t1 = first_token(a, r1);
    const bool some = r0 < r1 && t0 < t1;
    return {r0, t0, some ? t1 - t0 : 0, 0, some ? bounded(a.prefix[g], 0, a.max_len) : 0};
}
__device__ __forceinline__ Segment own_of(const KvCache &c, const KvAttendShared &a, const SharedPlan &pl, int row) {
    const int t0 = first_token(a, row), t1 = first_token(a, row + 1);
    return {row, t0, max(t1 - t0, 0), pl.row_prefix[row], kv_len(a.lens, row, a.max_len)};
}
__device__ __forceinline__ int blocks_of(const Segment &s, int group, int lines) {
    return (int)(((int64_t)s.tokens * group + lines - 1) / lines);
}
__device__ __forceinline__ int chunks_of(const Segment &s) {
    return s.tokens > 0 && s.end > s.start ? (s.end - s.start + UNIT - 1) / UNIT : 0;
}

// The first `count` workgroups of the launch find each token's row; the last one counts units.
constexpr int PLAN_THREADS = 256;
__global__ __launch_bounds__(PLAN_THREADS) void kv_shared_plan_kernel(KvCache c, KvAttendShared a, SharedPlan pl) {
    __shared__ int64_t s_wave[PLAN_THREADS / 64];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (blockIdx.x + 1 < gridDim.x) {
        const int token = blockIdx.x * PLAN_THREADS + tid;
        if (token >= a.tokens) return;
        int row = token, behind = 0;
        if (a.cu) {
            int low = 0, high = c.rows;  // the first row that ends past the token
            while (low < high) {
                const int mid = (low + high) / 2;
                if (a.cu[mid + 1] <= token) low = mid + 1;
                else high = mid;
            }
            row = low < c.rows && a.cu[low] <= token ? low : -1;
            if (row >= 0) behind = min(a.cu[row + 1], a.tokens) - 1 - token;
        }
        pl.token_row[token] = row;
        pl.token_sees[token] = row < 0 ? 0 : max(kv_len(a.lens, row, a.max_len) - behind, 0);
        return;
    }
    // Each row's group and prefix.
    for (int r = tid; r < c.rows; r += PLAN_THREADS) {
        int g = -1, p = 0;
        if (a.group_rows) {
            int low = 0, high = a.groups;
            while (low < high) {
                const int mid = (low + high) / 2;
                if (a.group_rows[mid + 1] <= r) low = mid + 1;
                else high = mid;
            }
            if (low < a.groups && a.group_rows[low] <= r) {
                g = low;
                p = bounded(a.prefix[g], 0, a.max_len);
            }
        }
        pl.row_group[r] = g;
        pl.row_prefix[r] = p;
    }
    __syncthreads();
    // Running sums of the segments' units, a strip of segments for each thread.
    for (int which = 0; which < 2; ++which) {
        const int n = which ? c.rows : a.groups;
        const int strip = (n + PLAN_THREADS - 1) / PLAN_THREADS, s0 = min(tid * strip, n), s1 = min(s0 + strip, n);
        auto units_of = [&](int s) {
            const Segment x = which ? own_of(c, a, pl, s) : prefix_of(c, a, s);
            return (int64_t)c.heads * blocks_of(x, pl.group, pl.side[which].lines) * chunks_of(x);
        };
        int64_t mine = 0;
        for (int s = s0; s < s1; ++s) mine += units_of(s);
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
            pl.side[which].units[s] = at;
            at += units_of(s);
        }
        if (tid == PLAN_THREADS - 1) pl.side[which].units[n] = upto;
        __syncthreads();
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
    return __builtin_bit_cast(u32x2_kv, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) i16x4_sh *)(uintptr_t)(uint32_t)(uintptr_t)lds));
}

// How a workgroup is made up, by head size and lines.
template <int DIM, int LW, int SW>
struct Shape {
    static constexpr int WAVES = LW * SW, THREADS = 64 * WAVES, LINES = 32 * LW;
    static constexpr int SUBS = SW == 1 && DIM < 256 ? 2 : 1;     // runs of 32 slots of a wave's tile
    static constexpr int TILE = 32 * SW * SUBS;                   // slots of a tile
    static constexpr int BUFS = SW == 1 ? 2 : 1;
    static constexpr int PIECES = DIM / 8;                        // of a row of a tile, 16 bytes each
    static constexpr int LOADS = TILE * PIECES / THREADS;         // of a thread, of keys and of values
    static constexpr int ROW = DIM * 2;
    static constexpr int PART = 32 * (DIM + 4) * 4;               // a wave's o, rows 16 bytes apart from a bank's turn
    static constexpr int BYTES = SW == 1 ? BUFS * 2 * TILE * ROW : std::max(BUFS * 2 * TILE * ROW, WAVES * PART);
};

template <int DIM, bool FP8, int LW, int SW>
__global__ __launch_bounds__(64 * LW * SW, DIM > 128 ? 1 : 2) void kv_shared_kernel(KvCache c, KvAttendShared a, SharedPlan pl,
                                                                                   int which) {
    using X = Shape<DIM, LW, SW>;
    constexpr int TILE = X::TILE, SUBS = X::SUBS, PIECES = X::PIECES, LOADS = X::LOADS, ROW = X::ROW;
    constexpr int ROWS_IN_BANKS = 256 / DIM;   // rows of a tile in 512 bytes, one turn of the banks
    constexpr int DB = DIM / 32, QF = DIM / 16;
    __shared__ __align__(16) uint8_t pool[X::BYTES];
    __shared__ int s_there[X::BUFS][TILE];
    __shared__ float s_m[X::WAVES][32], s_l[X::WAVES][32];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int half = lane >> 5, col = lane & 31;
    const int lw = wave % LW, sw = wave / LW;
    const auto &side = pl.side[which];
    const int segments = which ? c.rows : a.groups;
    const int64_t units = side.units[segments];
    const int shares = (int)min((int64_t)side.wgs, units);
    // Neighbouring shares, which meet the same keys, go to one XCD.
    const int share = side.wgs % 8 || shares < side.wgs ? (int)blockIdx.x : (int)(blockIdx.x % 8) * (side.wgs / 8) + (int)(blockIdx.x / 8);
    if (share >= shares) return;
    int64_t u = units * share / shares;
    const int64_t u1 = units * (share + 1) / shares;
    int seg = 0;  // segments that end at or before u
    for (int at = 0; at < segments; at += 64) {
        const int n = __popcll(__ballot(at + lane < segments && side.units[at + lane + 1] <= u));
        seg += n;
        if (n < 64) break;
    }

    // Where this thread's pieces of a tile go, and where its lane reads: within a row the
    // pieces' places are turned by the row's number.
    auto k_at = [&](int s, int piece) { return s * ROW + ((piece ^ ((s / ROWS_IN_BANKS) & (PIECES - 1))) << 4); };
    auto v_at = [&](int s, int piece) {
        return s * ROW + ((piece ^ (((s / ROWS_IN_BANKS) & (8 / ROWS_IN_BANKS - 1)) << 2)) << 4);
    };
    const int k_read = col * ROW, k_turn = (half ^ ((col / ROWS_IN_BANKS) & (PIECES - 1))) << 4;
    const int v_slot = 4 * half + (lane & 15) / 4;
    const int v_turn = (v_slot / ROWS_IN_BANKS) & (8 / ROWS_IN_BANKS - 1);
    const int v_read = v_slot * ROW + (2 * ((lane >> 4) & 1) + (lane & 3) / 2) * 16 + (lane & 1) * 8;

    for (;;) {  // a piece: chunks [c0, c1) of one block of a segment's lines
        const Segment sg = which ? own_of(c, a, pl, seg) : prefix_of(c, a, seg);
        const int chunks = chunks_of(sg), blocks = blocks_of(sg, pl.group, X::LINES);
        const int64_t in = u - side.units[seg];
        const int head = (int)(in / ((int64_t)blocks * chunks)), rest = (int)(in % ((int64_t)blocks * chunks));
        const int block = rest / chunks, c0 = rest % chunks, c1 = (int)min((int64_t)chunks, c0 + (u1 - u));
        const int nlines = sg.tokens * pl.group - block * X::LINES;  // of this block and those after it
        const int line = lw * 32 + col;
        const bool valid = line < nlines;
        const int seg_line = block * X::LINES + (valid ? line : 0);
        const int token = sg.token + seg_line / pl.group, q_head = head * pl.group + seg_line % pl.group;
        const int32_t *table = c.table + (int64_t)sg.row * c.table_ld;
        // The last slot that any line sees: a row's later tokens see more.
        int end = sg.end;
        if (which) {
            const int last = min(X::LINES, nlines) - 1 + block * X::LINES;
            end = min(end, pl.token_sees[sg.token + last / pl.group]);
        }
        const int from = sg.start + c0 * UNIT, to = min(sg.start + c1 * UNIT, end);
        const int tiles = to > from ? (to - from + TILE - 1) / TILE : 0;
        const int sees = valid ? min(pl.token_sees[token], end) : INT32_MAX;
        const int least = -wave_max(-sees), most = wave_max(valid ? sees : 0);

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
        const float by = fabsf(a.scale) * 1.44269504088896340736f * (FP8 ? c.k_scale[head] : 1.f);
        // Weights are up to 2^RAISE, and as many meet the values as the segment has slots: times a
        // power of two, in their exponent, they sum to 1 at the most, and finite values cannot run over.
        const int n = sg.end - sg.start;
        const float room = RAISE + (n > 1 ? 32 - __builtin_clz(n - 1) : 0);

        // A thread's pieces of a tile: the slot of its i-th one, that slot's page, and the bytes.
        auto slot_of = [&](int i) { return (tid + i * X::THREADS) / PIECES; };
        const int piece = tid % PIECES;
        int32_t page[LOADS];
        typedef typename std::conditional<FP8, u32x2_kv, u32x4_kv>::type Raw;
        Raw kr[LOADS], vr[LOADS];
        uint32_t ok = 0;  // bit i: the i-th piece's slot counts
        auto ask_pages = [&](int tile) {
#pragma unroll
            for (int i = 0; i < LOADS; ++i) page[i] = table[min(from + tile * TILE + slot_of(i), c.cap - 1) >> c.page_log2];
        };
        auto ask = [&](int tile) {
            ok = 0;
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int slot = from + tile * TILE + slot_of(i);
                const bool there = page[i] >= 0 && page[i] < c.pages;
                ok |= (uint32_t)(there && slot < to) << i;
                const int64_t at = ((((int64_t)(there ? page[i] : 0) * c.heads + head) << c.page_log2) +
                                    (slot & ((1 << c.page_log2) - 1))) * (FP8 ? DIM : DIM * 2) + piece * (FP8 ? 8 : 16);
                kr[i] = *reinterpret_cast<const Raw *>(c.k + at);
                vr[i] = *reinterpret_cast<const Raw *>(c.v + at);
            }
        };
        auto put = [&](int buf) {
            uint8_t *kb = pool + buf * 2 * TILE * ROW, *vb = kb + TILE * ROW;
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int s = slot_of(i);
                const bool there = ok >> i & 1;
                u32x4_kv k, v;
                if constexpr (FP8) {
                    k = u32x4_kv{fp8_widened<0>(kr[i][0]), fp8_widened<1>(kr[i][0]), fp8_widened<0>(kr[i][1]), fp8_widened<1>(kr[i][1])};
                    v = u32x4_kv{fp8_widened<0>(vr[i][0]), fp8_widened<1>(vr[i][0]), fp8_widened<0>(vr[i][1]), fp8_widened<1>(vr[i][1])};
                } else {
                    k = kr[i];
                    v = vr[i];
                }
                // 0 times what lies in a slot that does not count could be NaN
                *reinterpret_cast<u32x4_kv *>(kb + k_at(s, piece)) = k;
                *reinterpret_cast<u32x4_kv *>(vb + v_at(s, piece)) = there ? v : u32x4_kv{0, 0, 0, 0};
                if (piece == 0) s_there[buf][s] = there;
            }
        };

        f32x16_sh o[DB];
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
        float m = NEG_INF, sum = 0.f;

        auto use = [&](int tile, int buf) {
            const int first = from + tile * TILE + sw * SUBS * 32;  // the wave's slots
            if (first >= most) return;
            const uint8_t *kb = pool + buf * 2 * TILE * ROW + sw * SUBS * 32 * ROW, *vb = kb + TILE * ROW;
            f32x16_sh s[SUBS];
            uint32_t there[SUBS];
            bool full = first + SUBS * 32 <= least;
#pragma unroll
            for (int b = 0; b < SUBS; ++b) {
                there[b] = (uint32_t)__ballot(s_there[buf][(sw * SUBS + b) * 32 + col] != 0);
                full = full && there[b] == ~0u;
#pragma unroll
                for (int i = 0; i < 16; ++i) s[b][i] = 0.f;
#pragma unroll
                for (int f = 0; f < QF; ++f) {
                    const u32x4_kv kf = *reinterpret_cast<const u32x4_kv *>(kb + b * 32 * ROW + k_read + (k_turn ^ (f << 5)));
                    s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_sh, kf),
                                                                   __builtin_bit_cast(bf16x8_sh, q[f]), s[b], 0, 0, 0);
                }
            }
            if (!full) {
#pragma unroll
                for (int b = 0; b < SUBS; ++b)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = 8 * (i / 4) + 4 * half + i % 4;
                        s[b][i] = (there[b] >> j & 1) && first + b * 32 + j < sees ? s[b][i] : NEG_INF;
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
            float part = 0.f;
            // A line may not see a slot that others of the wave do: its weight is 0, but what lies
            // there may be NaN or infinite.
            bool careful = false;
            if (!full && least < min(first + SUBS * 32, end)) {
                bool odd = false;
                for (int i = lane; i < SUBS * 32 * PIECES; i += 64) {
                    const u32x4_kv x = *reinterpret_cast<const u32x4_kv *>(vb + i * 16);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        odd = odd || (x[e] & 0x7F80u) == 0x7F80u || (x[e] & 0x7F800000u) == 0x7F800000u;
                }
                careful = __any(odd);
            }
#pragma unroll
            for (int b = 0; b < SUBS; ++b) {
                uint32_t p[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s[b][2 * i] = __builtin_amdgcn_exp2f(fmaf(s[b][2 * i], by, -ref));
                    s[b][2 * i + 1] = __builtin_amdgcn_exp2f(fmaf(s[b][2 * i + 1], by, -ref));
                    p[i] = bf16_pair(s[b][2 * i], s[b][2 * i + 1]);
                    part = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_sh, p[i]),
                                                           bf16x2_sh{(__bf16)1.f, (__bf16)1.f}, part, false);
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const u32x4_kv pf = {p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]};
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const uint8_t *src = vb + (b * 32 + 16 * k) * ROW + v_read + ((d ^ v_turn) << 6);
                        const u32x2_kv v0 = transposed(src), v1 = transposed(src + 8 * ROW);
                        u32x4_kv vf = {v0[0], v0[1], v1[0], v1[1]};
                        if (careful) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                if ((vf[e] & 0x7F80u) == 0x7F80u) vf[e] &= 0xFFFF0000u;
                                if ((vf[e] & 0x7F800000u) == 0x7F800000u) vf[e] &= 0x0000FFFFu;
                            }
                        }
                        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_sh, vf),
                                                                       __builtin_bit_cast(bf16x8_sh, pf), o[d], 0, 0, 0);
                    }
                }
                if (careful) {
                    // What the product left out, for the lines that do see it, one slot after the other.
                    for (int j = 0; j < 32; ++j) {
                        float w = 0.f;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (8 * (i / 4) + i % 4 == (j & ~4)) w = s[b][i];
                        w = __shfl(w, col + 32 * (j >> 2 & 1));
                        const bool seen = first + b * 32 + j < sees;
#pragma unroll
                        for (int d = 0; d < DB; ++d)
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int dim = 32 * d + 8 * (i / 4) + 4 * half + i % 4;
                                const uint32_t x = *reinterpret_cast<const uint16_t *>(vb + v_at(b * 32 + j, dim / 8) + dim % 8 * 2);
                                if ((x & 0x7F80u) == 0x7F80u && seen) o[d][i] += w * __uint_as_float(x << 16);
                            }
                    }
                }
            }
            sum += part;
        };

        if (tiles > 0) {
            ask_pages(0);
            ask(0);
            if constexpr (X::BUFS == 2) {
                ask_pages(min(1, tiles - 1));
                put(0);
                ask(min(1, tiles - 1));
                ask_pages(min(2, tiles - 1));
                __syncthreads();
                for (int t = 0; t < tiles; ++t) {
                    use(t, t & 1);
                    if (t + 1 < tiles) {
                        put((t + 1) & 1);
                        ask(min(t + 2, tiles - 1));
                        ask_pages(min(t + 3, tiles - 1));
                    }
                    __syncthreads();
                }
            } else {
                ask_pages(min(1, tiles - 1));
                for (int t = 0; t < tiles; ++t) {
                    put(0);
                    ask(min(t + 1, tiles - 1));
                    ask_pages(min(t + 2, tiles - 1));
                    __syncthreads();
                    use(t, 0);
                    __syncthreads();
                }
            }
        }

        // The piece's result.  One that has all that its lines see is the result; others wait for the join.
        sum += __shfl_xor(sum, 32);
        const bool sole = which && sg.start == 0 && c0 == 0 && c1 == chunks;
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
        if constexpr (SW == 1) {
            if (valid)
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 16; i += 4)
                        store(line, 32 * d + 2 * i + 4 * half, f32x4_sh{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]}, m, sum);
        } else {
            float *mine = reinterpret_cast<float *>(pool) + wave * (X::PART / 4) + col * (DIM + 4);
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                    *reinterpret_cast<f32x4_sh *>(mine + 32 * d + 2 * i + 4 * half) = f32x4_sh{o[d][i], o[d][i + 1], o[d][i + 2], o[d][i + 3]};
            if (half == 0) {
                s_m[wave][col] = m;
                s_l[wave][col] = sum;
            }
            __syncthreads();
            for (int i = tid; i < min(X::LINES, nlines) * (DIM / 4); i += X::THREADS) {
                const int ln = i / (DIM / 4), d = i % (DIM / 4) * 4;
                float top = NEG_INF, total = 0.f;
                f32x4_sh x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < SW; ++w) top = fmaxf(top, s_m[w * LW + ln / 32][ln % 32]);
#pragma unroll
                for (int w = 0; w < SW; ++w) {
                    const int v = w * LW + ln / 32;
                    const float mw = s_m[v][ln % 32], f = mw == top ? 1.f : __builtin_amdgcn_exp2f(mw - top);
                    total += s_l[v][ln % 32] * f;
                    x += *reinterpret_cast<const f32x4_sh *>(reinterpret_cast<const float *>(pool) + v * (X::PART / 4) +
                                                             ln % 32 * (DIM + 4) + d) * f;
                }
                store(ln, d, x, top, total);
            }
        }
        u += c1 - c0;
        if (u >= u1) return;
        __syncthreads();  // pool and the sums are free
        while (side.units[seg + 1] <= u) ++seg;
    }
}

// The last launch: each line's parts, in a fixed order.
constexpr int JOIN_THREADS = 256;
template <int DIM>
__global__ __launch_bounds__(JOIN_THREADS) void kv_shared_join_kernel(KvCache c, KvAttendShared a, SharedPlan pl) {
    constexpr int LANES = DIM / 4;  // of a line, four dims each
    const int64_t which_line = (int64_t)blockIdx.x * (JOIN_THREADS / LANES) + threadIdx.x / LANES;
    if (which_line >= (int64_t)a.tokens * a.q_heads) return;
    const int token = (int)(which_line / a.q_heads), qh = (int)(which_line % a.q_heads), d = threadIdx.x % LANES * 4;
    const int row = pl.token_row[token];
    if (row < 0) return;
    const int head = qh / pl.group;
    int first[2] = {0, 0}, n[2] = {0, 0}, line[2] = {0, 0};  // of each side: the first part's workgroup, parts, line of its block
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const int seg = which ? row : pl.row_group[row];
        if (seg < 0) continue;
        const auto &side = pl.side[which];
        const Segment sg = which ? own_of(c, a, pl, seg) : prefix_of(c, a, seg);
        const int chunks = chunks_of(sg);
        if (chunks == 0) continue;
        const int64_t units = side.units[which ? c.rows : a.groups];
        const int shares = (int)min((int64_t)side.wgs, units);
        const int in = (token - sg.token) * pl.group + qh % pl.group, block = in / side.lines;
        const int64_t at = side.units[seg] + ((int64_t)head * blocks_of(sg, pl.group, side.lines) + block) * chunks;
        first[which] = owner_of(at, units, shares);
        n[which] = owner_of(at + chunks - 1, units, shares) - first[which] + 1;
        line[which] = in % side.lines;
        if (which && sg.start == 0 && n[1] == 1) return;  // written already
    }
    auto place = [&](int i, const float *&ml, const float *&po) {
        const int which = i >= n[0];
        const auto &side = pl.side[which];
        i -= which ? n[0] : 0;
        const int64_t at = i == 0 ? which_line : (int64_t)(first[which] + i) * side.lines + line[which];
        ml = (i == 0 ? side.first_ml : side.more_ml) + 2 * at;
        po = (i == 0 ? side.first_o : side.more_o) + at * DIM + d;
    };
    const int parts = n[0] + n[1];
    float top = NEG_INF, total = 0.f;
    for (int i = 0; i < parts; ++i) {
        const float *ml, *po;
        place(i, ml, po);
        const float m = ml[0], up = fmaxf(top, m);
        total = total * (top == up ? 1.f : __builtin_amdgcn_exp2f(top - up)) + ml[1] * (m == up ? 1.f : __builtin_amdgcn_exp2f(m - up));
        top = up;
    }
    // Each part's share of the sum first: finite values cannot run over.
    const float inv = total == 0.f ? 0.f : 1.f / total;
    f32x4_sh x = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < parts; ++i) {
        const float *ml, *po;
        place(i, ml, po);
        const float m = ml[0];
        x += *reinterpret_cast<const f32x4_sh *>(po) * ((m == top ? 1.f : __builtin_amdgcn_exp2f(m - top)) * inv);
    }
    if (total == 0.f) x = f32x4_sh{0.f, 0.f, 0.f, 0.f};  // nothing to attend to, whatever the values are
    if (c.fp8) x *= c.v_scale[head];
    *reinterpret_cast<u32x2_kv *>(a.out + (int64_t)token * a.out_ld + (int64_t)qh * DIM + d) =
        u32x2_kv{bf16_pair(x[0], x[1]), bf16_pair(x[2], x[3])};
}

// The plan, its scratch laid out from `base`; returns the bytes (-1: more than a launch takes).
static int64_t shared_plan(const KvCache &c, int q_heads, int tokens, int groups, int max_len, int cu_count, uint8_t *base,
                           SharedPlan *pl) {
    pl->group = q_heads / c.heads;
    const int64_t lines = (int64_t)tokens * pl->group, chunks = (max_len + UNIT - 1) / UNIT;
    for (int which = 0; which < 2; ++which) {
        auto &side = pl->side[which];
        const int64_t segments = which ? c.rows : groups;
        const int64_t mean = segments ? (lines + segments - 1) / segments : 0;  // lines of a segment
        side.lines = mean <= 32 ? 32 : mean <= 64 ? 64 : 128;
        const int64_t most = segments ? (lines / side.lines + segments) * c.heads * chunks : 0;
        if (most > INT32_MAX) return -1;
        side.wgs = (int)std::min<int64_t>(most, (int64_t)cu_count * (c.dim > 128 ? 1 : 2));
    }
    if (!fits_launch((int64_t)tokens * q_heads, JOIN_THREADS)) return -1;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        uint8_t *p = base ? base + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    pl->token_row = (int32_t *)take((int64_t)tokens * 4);
    pl->token_sees = (int32_t *)take((int64_t)tokens * 4);
    pl->row_prefix = (int32_t *)take((int64_t)c.rows * 4);
    pl->row_group = (int32_t *)take((int64_t)c.rows * 4);
    for (int which = 0; which < 2; ++which) {
        auto &side = pl->side[which];
        const int64_t all = side.wgs ? (int64_t)tokens * q_heads : 0, more = (int64_t)side.wgs * side.lines;
        side.units = (int64_t *)take(((int64_t)(which ? c.rows : groups) + 1) * 8);
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

template <int DIM, bool FP8>
static void launch_shared(const KvCache &c, const KvAttendShared &a, const SharedPlan &pl, hipStream_t stream) {
    for (int which = 0; which < 2; ++which) {
        const auto &side = pl.side[which];
        const dim3 grid((unsigned)side.wgs);
        if (side.wgs == 0) continue;
        if (side.lines == 32) hipLaunchKernelGGL((kv_shared_kernel<DIM, FP8, 1, 4>), grid, dim3(256), 0, stream, c, a, pl, which);
        else if (side.lines == 64) hipLaunchKernelGGL((kv_shared_kernel<DIM, FP8, 2, 2>), grid, dim3(256), 0, stream, c, a, pl, which);
        else hipLaunchKernelGGL((kv_shared_kernel<DIM, FP8, 4, 1>), grid, dim3(256), 0, stream, c, a, pl, which);
    }
    const int64_t lines = (int64_t)a.tokens * a.q_heads;
    constexpr int EACH = JOIN_THREADS / (DIM / 4);
    hipLaunchKernelGGL((kv_shared_join_kernel<DIM>), dim3((unsigned)((lines + EACH - 1) / EACH)), dim3(JOIN_THREADS), 0, stream,
                       c, a, pl);
}

hipError_t launch_kv_attend_shared(const KvCache &c, const KvAttendShared &a, int cu_count, hipStream_t stream) {
    SharedPlan pl;
    shared_plan(c, a.q_heads, a.tokens, a.groups, a.max_len, cu_count, a.ws, &pl);
    const unsigned finders = (unsigned)((a.tokens + PLAN_THREADS - 1) / PLAN_THREADS);
    hipLaunchKernelGGL(kv_shared_plan_kernel, dim3(finders + 1), dim3(PLAN_THREADS), 0, stream, c, a, pl);
    switch (c.dim) {
    case 64: if (c.fp8) launch_shared<64, true>(c, a, pl, stream); else launch_shared<64, false>(c, a, pl, stream); break;
    case 128: if (c.fp8) launch_shared<128, true>(c, a, pl, stream); else launch_shared<128, false>(c, a, pl, stream); break;
    default: if (c.fp8) launch_shared<256, true>(c, a, pl, stream); else launch_shared<256, false>(c, a, pl, stream); break;
    }
    return hipGetLastError();
}

}  // namespace nbw
