// verify.hip -- which drafted tokens stand, and the token after them, gfx950.
//
// The drafts of a row are looked at side by side: a lane gathers p[x] and q[x] of
// one, and the first that is refused ends the row's run.  u q < p in fp64 is exact,
// the product of two numbers of 24 bits having 48.
//
// The next token is found in the running sum of one line's weights, max(p - q, 0) or p.
// A first launch sums spans of 1024 of them, a wave a span, or a few one after the other where
// there are more than run at once; a second one, a wave a row, finds the span in which the sum passes
// u times the whole, and then the place in it.  Nothing is shared between waves, so there is no barrier.
// (A few short rows: a workgroup each, both in one launch, with a barrier between.)
// Sums are in fp64 and in a fixed order: of 128 thousand weights they are off by about 1e-14, so that the
// place is the exact one but for one draw in 1e9.
//
// Bound: memory, one line a row, or two where a draft was refused; for few rows the
// chain of loads (cu -> tokens -> p, q -> line) and the second launch.  One row of 32000 weights 6.8 us,
// 64 rows of 128000 (56 MB) 11.4 + 4.5, 256 lines of 160001 in bf16 (82 MB) 17.4 + 4.7: 4.7 TB/s, held up
// by the arithmetic of the weights.  (A workgroup a span, with barriers: 12.3 us for one row, 43 for the 256 lines; 32 weights a
// lane 28 in place of 25, loads at shifted, aligned addresses 27, six waves a SIMD 26.)
#include <algorithm>

#include "kv.h"

namespace nbw {

constexpr int VERIFY_THREADS = 256;
constexpr int EACH = 16;         // weights of a lane
constexpr int SPAN = 64 * EACH;  // of a wave

// A row's lines.
struct Lines {
    int first, count;
};
__device__ __forceinline__ Lines lines_of(const VerifyDrafts &a, int row) {
    if (!a.cu) return {row, 1};
    const int first = min(max(a.cu[row], 0), a.tokens), end = min(max(a.cu[row + 1], first), a.tokens);
    return {first, end - first};
}

template <bool BF16>
__device__ __forceinline__ float prob(const void *p, int64_t i) {
    if constexpr (BF16) return __uint_as_float((uint32_t)((const uint16_t *)p)[i] << 16);
    else return ((const float *)p)[i];
}

// How many of a row's drafts stand; the same in all lanes.
template <bool BF16>
__device__ __forceinline__ int standing(const VerifyDrafts &a, const Lines &l) {
    const int lane = threadIdx.x & 63;
    for (int i0 = 0; i0 < l.count - 1; i0 += 64) {
        const int i = i0 + lane;
        bool stands = false;
        if (i < l.count - 1) {
            const int64_t t = l.first + i;
            const int x = a.ids[t + 1];
            if (x >= 0 && x < a.vocab) {
                const double p = prob<BF16>(a.target, t * a.target_ld + x);
                const double q = a.draft ? (double)prob<BF16>(a.draft, t * a.draft_ld + x) : 1.0;
                stands = (double)a.u[t] * q < p;
            }
        }
        const unsigned long long refused = ~__ballot(stands);
        if (refused) return min(i0 + __builtin_ctzll(refused), l.count - 1);
    }
    return l.count - 1;
}

// A line's weights.
template <bool BF16>
struct Line {
    const void *target, *draft;  // draft: null if p alone counts
    int64_t p0, q0;              // the line's first element in each
    int vocab, out;              // the one token whose weight is 0 (-1: none)

    static constexpr int N = BF16 ? 8 : 4;  // in 16 bytes

    // What p - q counts as: itself, in fp64, if it is positive and finite, else 0.
    __device__ __forceinline__ double weight(int i, float p, float q) const {
        const float inf = __builtin_inff();
        const bool counts = p > q && p < inf && q > -inf && i != out;
        return (double)(counts ? p : 0.f) - (double)(counts ? q : 0.f);
    }
    __device__ __forceinline__ static float get(const u32x4_kv &w, int i) {
        if constexpr (BF16) return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
        else return __uint_as_float(w[i]);
    }
    // use(p, q) for a lane's elements of a whole span, a wave's loads side by side.
    template <bool DRAFT, class F>
    __device__ __forceinline__ void raw(int64_t at, F use) const {
        constexpr int PACKS = EACH / N, SIZE = BF16 ? 2 : 4;
        u32x4_kv p[PACKS], q[PACKS];  // at any address: no more aligned than an element
        const int64_t i = at + (threadIdx.x & 63) * N;
#pragma unroll
        for (int k = 0; k < PACKS; ++k) {
            __builtin_memcpy(&p[k], (const uint8_t *)target + (p0 + i + k * 64 * N) * SIZE, 16);
            if (DRAFT) __builtin_memcpy(&q[k], (const uint8_t *)draft + (q0 + i + k * 64 * N) * SIZE, 16);
        }
#pragma unroll
        for (int k = 0; k < PACKS; ++k)
#pragma unroll
            for (int e = 0; e < N; ++e) use(get(p[k], e), DRAFT ? get(q[k], e) : 0.f);
    }
    // use(i, weight) for a lane's weights of span `span`, in packs of N: pack k begins at
    // k * STEP + lane * FIRST within the span.
    template <int STEP, int FIRST, class F>
    __device__ __forceinline__ void weights(int span, F use) const {
        constexpr int PACKS = EACH / N;
        const int64_t at = (int64_t)span * SPAN;
        const int mine = (threadIdx.x & 63) * FIRST;
        if (at + SPAN <= vocab) {
            u32x4_kv p[PACKS], q[PACKS];  // at any address: no more aligned than an element
#pragma unroll
            for (int k = 0; k < PACKS; ++k) {
                const int64_t i = at + mine + k * STEP;
                __builtin_memcpy(&p[k], (const uint8_t *)target + (p0 + i) * (BF16 ? 2 : 4), 16);
                if (draft) __builtin_memcpy(&q[k], (const uint8_t *)draft + (q0 + i) * (BF16 ? 2 : 4), 16);
                else q[k] = u32x4_kv{0, 0, 0, 0};
            }
#pragma unroll
            for (int k = 0; k < PACKS; ++k)
#pragma unroll
                for (int e = 0; e < N; ++e)
                    use(k * N + e, weight((int)at + mine + k * STEP + e, get(p[k], e), get(q[k], e)));
        } else {
#pragma unroll
            for (int k = 0; k < PACKS; ++k)
#pragma unroll
                for (int e = 0; e < N; ++e) {
                    const int64_t i = at + mine + k * STEP + e;
                    const bool there = i < vocab;
                    use(k * N + e, there ? weight((int)i, prob<BF16>(target, p0 + i), draft ? prob<BF16>(draft, q0 + i) : 0.f) : 0.0);
                }
        }
    }
};
template <bool BF16>
__device__ __forceinline__ Line<BF16> line_of(const VerifyDrafts &a, const Lines &l, int stands) {
    const int64_t t = l.first + stands;
    const bool refused = stands < l.count - 1;
    return {a.target, refused ? a.draft : nullptr, t * a.target_ld, t * a.draft_ld, a.vocab,
            refused && !a.draft ? a.ids[t + 1] : -1};
}

// Sums of fp64 over this lane and those before it, in register-to-register steps (as wave_running).
template <int CTRL, int ROWS>
__device__ __forceinline__ double from_lane64(double x) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = (uint32_t)from_lane<CTRL, ROWS>(0, (int32_t)(uint32_t)b), hi = (uint32_t)from_lane<CTRL, ROWS>(0, (int32_t)(b >> 32));
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double running_sum(double x) {
    x += from_lane64<0x111, 0xF>(x);
    x += from_lane64<0x112, 0xF>(x);
    x += from_lane64<0x114, 0xF>(x);
    x += from_lane64<0x118, 0xF>(x);
    x += from_lane64<0x142, 0xA>(x);
    return x + from_lane64<0x143, 0xC>(x);
}
__device__ __forceinline__ double at_lane(double x, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, x);
    const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)b, lane), hi = __builtin_amdgcn_readlane((uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <bool BF16>
__device__ __forceinline__ double span_sum(const Line<BF16> &line, int span) {
    double w = 0.0;
    const int64_t at = (int64_t)span * SPAN;
    // In a whole span without the token left out a weight is max(p - q, 0), a NaN giving 0; only should the sum not
    // be finite is each looked at.  (The arithmetic of a weight decides: 256 lines of 160001 25 us with
    // all its comparisons, 19 so.)
    if (at + SPAN <= line.vocab && (line.out < at || line.out >= at + SPAN)) {
        if (line.draft) line.template raw<true>(at, [&](float p, float q) { w += fmax((double)p - (double)q, 0.0); });
        else line.template raw<false>(at, [&](float p, float) { w += (double)fmaxf(p, 0.f); });
        w = at_lane(running_sum(w), 63);
        if (w < __builtin_inf()) return w;
        w = 0.0;
    }
    // a wave's loads side by side
    line.template weights<64 * Line<BF16>::N, Line<BF16>::N>(span, [&](int, double x) { w += x; });
    return at_lane(running_sum(w), 63);
}

// The first launch: the sums of each row's spans, `run` of them to a wave.
template <bool BF16>
__global__ __launch_bounds__(VERIFY_THREADS) void verify_sums_kernel(VerifyDrafts a, int spans, int run, double *sums) {
    const int runs = (spans + run - 1) / run;
    const int wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * (VERIFY_THREADS / 64) + (threadIdx.x >> 6)));
    const int row = wave / runs, first = wave % runs * run;
    if (row >= a.rows) return;
    const bool one = (threadIdx.x & 63) == 0;
    const Lines l = lines_of(a, row);
    if (l.count <= 0) {
        if (first == 0 && one) a.accepted[row] = 0;
        return;
    }
    const int stands = standing<BF16>(a, l);
    if (first == 0 && one) a.accepted[row] = stands;
    const Line<BF16> line = line_of<BF16>(a, l, stands);
    for (int s = first; s < min(first + run, spans); ++s) {
        const double w = span_sum(line, s);
        if (one) sums[(int64_t)row * spans + s] = w;
    }
}

// A row's next token from its spans' sums, by a wave.  A lane keeps the sums of KEPT spans, of 64 of them each; `mine`
// has all of them.
template <bool BF16, int KEPT>
__device__ __forceinline__ void pick_next(const VerifyDrafts &a, int row, const Lines &l, int stands, int spans,
                                          const double (&kept)[KEPT], const double *mine) {
    const int lane = threadIdx.x & 63;
    Line<BF16> line = line_of<BF16>(a, l, stands);
    const float u32 = a.u[l.first + l.count - 1];
    const double u = u32 > 0.f ? (u32 < 1.f ? (double)u32 : 1.0) : 0.0;
    bool again = false;  // no difference is above 0: p itself, whose sums are formed here
    auto sums_from = [&](int s0) {  // 64 spans' sums from s0 on, one in each lane
        if (!again) {
            if (s0 < KEPT * 64) {
                double x = 0.0;
#pragma unroll
                for (int i = 0; i < KEPT; ++i) x = i * 64 == s0 ? kept[i] : x;
                return x;
            }
            return mine && s0 + lane < spans ? mine[s0 + lane] : 0.0;
        }
        double x = 0.0;
        for (int s = s0; s < min(s0 + 64, spans); ++s) {
            const double w = span_sum(line, s);
            x = s - s0 == lane ? w : x;
        }
        return x;
    };
    double all = 0.0;
    for (int pass = 0; pass < 2 && all == 0.0; ++pass) {
        if (pass == 1) {
            again = true;
            line.draft = nullptr;
            line.out = -1;
        }
        for (int s0 = 0; s0 < spans; s0 += 64) all += at_lane(running_sum(sums_from(s0)), 63);
    }
    if (all == 0.0) {
        if (lane == 0) a.next[row] = -1;
        return;
    }
    const double goal = u * all;
    // The first span whose end is past the goal; should rounding leave none, the last that has any weight.
    int span = -1;
    double lead = 0.0, before = 0.0;
    for (int s0 = 0; s0 < spans; s0 += 64) {
        const double x = sums_from(s0), upto = running_sum(x);
        const unsigned long long some = __ballot(x > 0.0), past = __ballot(x > 0.0 && lead + upto > goal);
        if (some) {
            const int at = past ? __builtin_ctzll(past) : 63 - __builtin_clzll(some);
            span = s0 + at;
            before = lead + at_lane(upto - x, at);
        }
        if (past) break;
        lead += at_lane(upto, 63);
    }
    // The same in the span, of which a lane has its weights in a row.
    double w[EACH], x = 0.0;
    line.template weights<Line<BF16>::N, EACH>(span, [&](int i, double v) {
        w[i] = v;
        x += v;
    });
    double at = before + (running_sum(x) - x);
    int pick = -1, last = -1;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        at += w[i];
        if (w[i] > 0.0) {
            last = i;
            if (pick < 0 && at > goal) pick = i;
        }
    }
    const unsigned long long picked = __ballot(pick >= 0), some = __ballot(last >= 0);
    const int from = picked ? __builtin_ctzll(picked) : 63 - __builtin_clzll(some);
    if (lane == from) a.next[row] = span * SPAN + lane * EACH + (picked ? pick : last);
}

// The second launch: each row's next token.
template <bool BF16>
__global__ __launch_bounds__(64) void verify_next_kernel(VerifyDrafts a, int spans, const double *sums) {
    const int row = blockIdx.x, lane = threadIdx.x;
    const double *const mine = sums + (int64_t)row * spans;
    constexpr int KEPT = 4;
    double kept[KEPT];
#pragma unroll
    for (int i = 0; i < KEPT; ++i) kept[i] = i * 64 + lane < spans ? mine[i * 64 + lane] : 0.0;
    const int stands = a.accepted[row];
    const Lines l = lines_of(a, row);
    if (l.count <= 0) {
        if (lane == 0) a.next[row] = -1;
        return;
    }
    pick_next<BF16>(a, row, l, stands, spans, kept, mine);
}

// Both in one launch, a workgroup a row, for few rows of few spans.
constexpr int ROW_WAVES = 16, ROW_SPANS = 64;
template <bool BF16>
__global__ __launch_bounds__(64 * ROW_WAVES) void verify_row_kernel(VerifyDrafts a, int spans) {
    __shared__ double s_sums[ROW_SPANS];
    const int row = blockIdx.x, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    const Lines l = lines_of(a, row);
    if (l.count <= 0) {
        if (threadIdx.x == 0) {
            a.accepted[row] = 0;
            a.next[row] = -1;
        }
        return;
    }
    const int stands = standing<BF16>(a, l);
    if (threadIdx.x == 0) a.accepted[row] = stands;
    const Line<BF16> line = line_of<BF16>(a, l, stands);
    for (int s = wave; s < spans; s += ROW_WAVES) {
        const double w = span_sum(line, s);
        if (lane == 0) s_sums[s] = w;
    }
    __syncthreads();
    if (wave) return;
    const double kept[1] = {lane < spans ? s_sums[lane] : 0.0};
    pick_next<BF16>(a, row, l, stands, spans, kept, nullptr);
}

static int spans_of(int vocab) { return (int)(((int64_t)vocab + SPAN - 1) / SPAN); }

int64_t verify_drafts_workspace_bytes(int rows, int vocab) {
    const int64_t spans = (int64_t)rows * spans_of(vocab);
    return fits_launch(spans, 64) ? spans * 8 : -1;
}

hipError_t launch_verify_drafts(const VerifyDrafts &a, int cu_count, hipStream_t stream) {
    const int spans = spans_of(a.vocab);
    // A workgroup a row spares a launch where a row is short and there is a CU for each.  Calls in one launch and in two (fp32, drafts
    // sampled): 1 row of 32000 8.8 and 11.6 us, of 65536 8.8 and 11.6, of 100000 9.5 and 11.6, of 128256 11.5 and 11.5, of 151936
    // 14.3 and 11.6, 64 of 100000 14.5 and 11.7, of 128256 18.0 and 14.8; 256 of 32000 11.5 and 14.2, of 65536 17.4 and 20.8; in bf16 256 of 65536 9.6 and
    // 12.5, 257 15.7 and 13.3.
    if (spans <= ROW_SPANS && a.rows <= cu_count) {
        const dim3 grid((unsigned)a.rows), threads(64 * ROW_WAVES);
        if (a.bf16) hipLaunchKernelGGL(verify_row_kernel<true>, grid, threads, 0, stream, a, spans);
        else hipLaunchKernelGGL(verify_row_kernel<false>, grid, threads, 0, stream, a, spans);
        return hipGetLastError();
    }
    // As many waves as run at once, 16 on a CU, each then with the same drafts to look at for several spans.
    const int64_t most = (int64_t)cu_count * 16;
    const int run = (int)std::min<int64_t>(spans, ((int64_t)a.rows * spans + most - 1) / most);
    const int64_t waves = (int64_t)a.rows * ((spans + run - 1) / run);
    const dim3 grid((unsigned)((waves + VERIFY_THREADS / 64 - 1) / (VERIFY_THREADS / 64))), threads(VERIFY_THREADS);
    if (a.bf16) {
        hipLaunchKernelGGL(verify_sums_kernel<true>, grid, threads, 0, stream, a, spans, run, (double *)a.ws);
        hipLaunchKernelGGL(verify_next_kernel<true>, dim3((unsigned)a.rows), dim3(64), 0, stream, a, spans, (const double *)a.ws);
    } else {
        hipLaunchKernelGGL(verify_sums_kernel<false>, grid, threads, 0, stream, a, spans, run, (double *)a.ws);
        hipLaunchKernelGGL(verify_next_kernel<false>, dim3((unsigned)a.rows), dim3(64), 0, stream, a, spans, (const double *)a.ws);
    }
    return hipGetLastError();
}

}  // namespace nbw
