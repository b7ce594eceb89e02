// kv_reserve.hip -- pages for the rows' next tokens and each token's place, gfx950.
//
// Everything follows from three running sums over the rows: pages given back,
// pages taken and tokens.  The i-th page taken is the i-th given back, or with
// none left free[count - 1 - (i - back)], so nothing has to pass from one
// workgroup to another: each forms the sums of all rows by itself, in LDS, and
// then does its share of the tokens and pages, finding the row of each by a
// search in the sums.  No entry that one workgroup reads is written by another.
//
// Rows are dealt out as SEGMENTS equal runs.  Up to that many rows a run is one
// row, and what a token needs to know of its row is in LDS; with more a search
// ends in a walk through a run.
//
// Bound: the chain of loads (lengths -> sums -> page numbers -> stores) of one
// launch: 3.5 us for one row, 6.5 for 256 rows with up to 6 tokens each, 6.8 for 96 prompts of up to
// 8192 tokens (4.8 MB written); a call takes 9 us with the host's checks of its tensors.
#include <algorithm>

#include "kv.h"

namespace nbw {

constexpr int RESERVE_THREADS = 256;
constexpr int SEGMENTS = 1024;
constexpr int OWN = SEGMENTS / RESERVE_THREADS;  // runs of one thread
constexpr uint32_t MOST = 0x7FFFFFFFu;           // sums stay at this once they reach it

// Running sums of one row or of all before it.
struct Sums {
    uint32_t back, take, tokens;
};
__device__ __forceinline__ uint32_t plus(uint32_t a, uint32_t b) { return min(a + b, MOST); }  // of two up to MOST
__device__ __forceinline__ Sums plus(const Sums &a, const Sums &b) {
    return {plus(a.back, b.back), plus(a.take, b.take), plus(a.tokens, b.tokens)};
}

// What a row holds and asks for.
struct Row {
    int len, held, need;
    Sums own;
};
__device__ __forceinline__ Row row_of(const KvCache &c, const KvReserve &a, int r) {
    Row x;
    x.len = kv_len(a.lens, r, c.cap);
    x.held = min(max(a.held[r], 0), c.width);
    const int want = max(a.want[r], 0), tokens = want <= c.cap - x.len ? want : 0;
    const int mask = (1 << c.page_log2) - 1;
    x.need = (int)(((int64_t)x.len + tokens + mask) >> c.page_log2);
    if (a.shared) x.need = max(x.need, min(a.shared[r], x.held));
    x.own = {(uint32_t)max(x.held - x.need, 0), (uint32_t)max(x.need - x.held, 0), (uint32_t)tokens};
    return x;
}

__global__ __launch_bounds__(RESERVE_THREADS) void kv_reserve_kernel(KvCache c, KvReserve a) {
    __shared__ uint32_t s_back[SEGMENTS], s_take[SEGMENTS], s_tokens[SEGMENTS];  // before each run
    __shared__ int32_t s_len[SEGMENTS], s_held[SEGMENTS], s_need[SEGMENTS];      // of runs of one row
    __shared__ Sums s_wave[RESERVE_THREADS / 64];
    __shared__ uint32_t s_first, s_granted[2];  // the first row that is not served; pages and tokens before it
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int run = (c.rows + SEGMENTS - 1) / SEGMENTS;  // rows of a run

    // The sums before every run.
    Sums mine[OWN], before = {0, 0, 0};
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int s = tid * OWN + i;
        mine[i] = {0, 0, 0};
        for (int r = s * run; r < min((s + 1) * run, c.rows); ++r) {
            const Row x = row_of(c, a, r);
            mine[i] = plus(mine[i], x.own);
            s_len[s] = x.len;
            s_held[s] = x.held;
            s_need[s] = x.need;
        }
        before = plus(before, mine[i]);
    }
    auto add = [](int32_t x, int32_t y) { return (int32_t)plus((uint32_t)x, (uint32_t)y); };
    Sums upto = {(uint32_t)wave_running((int32_t)before.back, 0, add), (uint32_t)wave_running((int32_t)before.take, 0, add),
                 (uint32_t)wave_running((int32_t)before.tokens, 0, add)};
    if (lane == 63) s_wave[wave] = upto;
    if (tid == 0) s_first = (uint32_t)c.rows;
    // What lies before this lane: the lane below's sums, and the waves' before this one.
    upto.back = __shfl_up(upto.back, 1);
    upto.take = __shfl_up(upto.take, 1);
    upto.tokens = __shfl_up(upto.tokens, 1);
    if (lane == 0) upto = {0, 0, 0};
    __syncthreads();
    Sums all = {0, 0, 0};
#pragma unroll
    for (int w = 0; w < RESERVE_THREADS / 64; ++w) {
        if (w < wave) upto = plus(s_wave[w], upto);
        all = plus(all, s_wave[w]);
    }
    const uint32_t count = (uint32_t)min(max(a.count[0], 0), a.free_size), back = all.back;
    const uint32_t spare = plus(count, back);
    auto fits = [&](const Sums &x) { return x.take < MOST && x.take <= spare && x.tokens <= (uint32_t)a.max_tokens; };

    // Rows are served up to the first that does not fit: sums only grow, so the run that
    // holds it is the first whose own end does not fit.
    Sums at = upto;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int s = tid * OWN + i;
        s_back[s] = at.back;
        s_take[s] = at.take;
        s_tokens[s] = at.tokens;
        const Sums end = plus(at, mine[i]);
        if (fits(at) && !fits(end)) {
            Sums x = at;
            int r = s * run;
            for (;; ++r) {
                const Sums y = plus(x, run == 1 ? mine[i] : row_of(c, a, r).own);
                if (!fits(y)) break;
                x = y;
            }
            s_first = (uint32_t)r;
            s_granted[0] = x.take;
            s_granted[1] = x.tokens;
        }
        at = end;
    }
    __syncthreads();
    const int served = (int)s_first;
    const uint32_t taken = served < c.rows ? s_granted[0] : all.take, tokens = served < c.rows ? s_granted[1] : all.tokens;

    // The row that a running sum's element is in, and the sums before it.
    struct Found {
        int row;
        Sums before;
    };
    auto find = [&](const uint32_t *sums, uint32_t i, auto which) {
        int s = 0;
#pragma unroll
        for (int step = SEGMENTS / 2; step; step >>= 1)
            if (sums[s + step] <= i) s += step;
        Found f = {s * run, {s_back[s], s_take[s], s_tokens[s]}};
        if (run > 1)
            for (;;) {
                const Sums own = row_of(c, a, f.row).own, end = plus(f.before, own);
                if (i < which(end)) break;
                f.before = end;
                ++f.row;
            }
        return f;
    };
    auto known = [&](int r) {
        if (run > 1) return row_of(c, a, r);
        Row x;
        x.len = s_len[r];
        x.held = s_held[r];
        x.need = s_need[r];
        return x;
    };
    auto entry = [&](int r, int i) { return a.table + (int64_t)r * c.table_ld + i; };
    auto given = [&](uint32_t i) {  // the i-th page given back
        const Found f = find(s_back, i, [](const Sums &x) { return x.back; });
        return *entry(f.row, known(f.row).need + (int)(i - f.before.back));
    };
    auto page_taken = [&](uint32_t i) { return i < back ? given(i) : a.free[count - 1 - (i - back)]; };

    const int stride = gridDim.x * RESERVE_THREADS, first = blockIdx.x * RESERVE_THREADS + tid;
    for (int t = first; t < a.max_tokens; t += stride) {
        int32_t position = 0;
        int64_t slot = -1;
        if ((uint32_t)t < tokens) {
            const Found f = find(s_tokens, (uint32_t)t, [](const Sums &x) { return x.tokens; });
            const Row x = known(f.row);
            const int nth = t - (int)f.before.tokens, j = x.len + nth, p = j >> c.page_log2;
            const int32_t page = p < x.held ? *entry(f.row, p) : page_taken(f.before.take + (uint32_t)(p - x.held));
            position = (a.seen ? a.seen[f.row] : x.len) + nth;
            if (page >= 0 && page < c.pages) slot = ((int64_t)page << c.page_log2) + (j & ((1 << c.page_log2) - 1));
        }
        a.positions[t] = position;
        a.slots[t] = slot;
    }
    for (uint32_t i = (uint32_t)first; i < max(taken, back); i += (uint32_t)stride) {
        if (i < taken) {
            const Found f = find(s_take, i, [](const Sums &x) { return x.take; });
            *entry(f.row, known(f.row).held + (int)(i - f.before.take)) = page_taken(i);
        } else if (spare - 1 - i < (uint32_t)a.free_size) {
            a.free[spare - 1 - i] = given(i);
        }
    }
    // The rows' own results.
    if (blockIdx.x != gridDim.x - 1) return;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const int s = tid * OWN + i;
        Sums x = {s_back[s], s_take[s], s_tokens[s]};
        for (int r = s * run; r < min((s + 1) * run, c.rows); ++r) {
            const Row y = row_of(c, a, r);
            const bool ok = r < served;
            a.cu[r] = (int32_t)(ok ? x.tokens : tokens);
            a.granted[r] = ok ? (int32_t)y.own.tokens : 0;
            a.held_out[r] = ok || y.own.back ? y.need : y.held;
            x = plus(x, y.own);
        }
    }
    if (tid == 0) {
        a.cu[c.rows] = (int32_t)tokens;
        a.count_out[0] = (int32_t)min(spare - taken, (uint32_t)a.free_size);
    }
}

hipError_t launch_kv_reserve(const KvCache &c, const KvReserve &a, int cu_count, hipStream_t stream) {
    // A workgroup for each 256 tokens, or each 64 rows' pages if there are fewer, up to two on a CU: each starts with
    // the sums of all rows.
    const int64_t work = std::max<int64_t>((a.max_tokens + RESERVE_THREADS - 1) / RESERVE_THREADS, (c.rows + 63) / 64);
    const dim3 grid((unsigned)std::max<int64_t>(1, std::min<int64_t>(work, (int64_t)cu_count * 2)));
    hipLaunchKernelGGL(kv_reserve_kernel, grid, dim3(RESERVE_THREADS), 0, stream, c, a);
    return hipGetLastError();
}

}  // namespace nbw
