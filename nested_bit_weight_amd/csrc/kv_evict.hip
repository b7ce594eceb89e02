// kv_evict.hip -- eviction from the cache by accumulated attention weight,
// gfx950.
//
// The plain kernel: one workgroup takes one (row, head).  The budget-th largest
// key is found by counting: four passes of 8 bits over the keys, each narrowing
// the range to one bin.  Then the slots are walked in order, 256 at a time, with
// running counts of the equals kept so far, of the gaps below the budget and of
// the slots that move into them; gaps and movers of equal number are paired
// through the workspace, and the pairs' rows are copied.
//
// A move reads at or past the budget and writes below it, so moves never meet.
#include "kv.h"

namespace nbw {

constexpr int EVICT_THREADS = 256;

// Keys as unsigned numbers of the same order.  -0 and +0 are equal.
__device__ __forceinline__ uint32_t evict_key(float acc, int32_t pos, int32_t newest, const KvEvict &a) {
    if (pos < a.sink || (int64_t)pos > (int64_t)newest - a.recent) return 0xFF800000u;  // +inf
    if (acc != acc) return 0x007FFFFFu;                                                 // -inf
    const uint32_t u = __float_as_uint(acc == 0.f ? 0.f : acc);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// The number of threads below this one for which `yes`, and of all of them.
__device__ __forceinline__ int rank_of(bool yes, int *waves, int &all) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const unsigned long long m = __ballot(yes);
    int below = __popcll(m & ((1ull << lane) - 1));
    __syncthreads();
    if (lane == 0) waves[wave] = __popcll(m);
    __syncthreads();
    all = 0;
    for (int w = 0; w < EVICT_THREADS / 64; ++w) {
        if (w < wave) below += waves[w];
        all += waves[w];
    }
    return below;
}

__global__ __launch_bounds__(EVICT_THREADS) void kv_evict_kernel(KvCache c, KvEvict a) {
    __shared__ int hist[256];
    __shared__ int waves[EVICT_THREADS / 64];
    __shared__ int found[2];
    const int tid = threadIdx.x;
    const int row = blockIdx.x / c.heads, head = blockIdx.x % c.heads;
    const int n = kv_len(a.lens, row, a.max_len), b = a.budget;
    const int64_t base = (int64_t)blockIdx.x * c.cap;
    if (head == 0 && tid == 0) a.lens_out[row] = n < b ? n : b;
    if (n <= b) {
        for (int j = tid; j < n; j += EVICT_THREADS) {
            a.acc_out[base + j] = a.acc[base + j];
            a.pos_out[base + j] = a.pos[base + j];
        }
        return;
    }
    int32_t newest = INT32_MIN;
    for (int j = tid; j < n; j += EVICT_THREADS) newest = max(newest, a.pos[base + j]);
    for (int d = 1; d < 64; d <<= 1) newest = max(newest, __shfl_xor(newest, d));
    if ((tid & 63) == 0) waves[tid >> 6] = newest;
    __syncthreads();
    for (int w = 0; w < EVICT_THREADS / 64; ++w) newest = max(newest, waves[w]);

    uint32_t prefix = 0;  // the leading bits of the budget-th largest key
    int want = b;         // its place among the keys with those bits
    for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();
        hist[tid] = 0;
        __syncthreads();
        for (int j = tid; j < n; j += EVICT_THREADS) {
            const uint32_t key = evict_key(a.acc[base + j], a.pos[base + j], newest, a);
            if (shift == 24 || (key >> (shift + 8)) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
        }
        __syncthreads();
        if (tid == 0) {
            int bin = 255, above = 0;
            while (bin > 0 && above + hist[bin] < want) above += hist[bin--];
            found[0] = bin;
            found[1] = above;
        }
        __syncthreads();
        prefix = prefix << 8 | (uint32_t)found[0];
        want -= found[1];
    }
    // `prefix` is the key itself now, and `want` how many equal to it stay.
    const int most = a.max_len - b < b ? a.max_len - b : b;  // moves at the most
    int32_t *to = reinterpret_cast<int32_t *>(a.ws) + (int64_t)blockIdx.x * 2 * most, *of = to + most;
    int equals = 0, gaps = 0, movers = 0;
    for (int j0 = 0; j0 < n; j0 += EVICT_THREADS) {
        const int j = j0 + tid;
        const bool there = j < n;
        const uint32_t key = there ? evict_key(a.acc[base + j], a.pos[base + j], newest, a) : 0;
        int all;
        const bool equal = there && key == prefix;
        const int r = equals + rank_of(equal, waves, all);
        equals += all;
        const bool keep = there && (key > prefix || (equal && r < want));
        const bool gap = there && !keep && j < b, mover = keep && j >= b;
        const int rg = gaps + rank_of(gap, waves, all);
        gaps += all;
        if (gap) to[rg] = j;
        const int rm = movers + rank_of(mover, waves, all);
        movers += all;
        if (mover) of[rm] = j;
        if (keep && j < b) {
            a.acc_out[base + j] = a.acc[base + j];
            a.pos_out[base + j] = a.pos[base + j];
        }
    }
    __syncthreads();
    const int row_bytes = c.fp8 ? c.dim : c.dim * 2, vecs = row_bytes / 16;
    for (int i = tid; i < movers * vecs; i += EVICT_THREADS) {
        const int m = i / vecs, part = i % vecs;
        if (part == 0) {
            a.acc_out[base + to[m]] = a.acc[base + of[m]];
            a.pos_out[base + to[m]] = a.pos[base + of[m]];
        }
        const int64_t src = kv_row(c, row, head, of[m]), dst = kv_row(c, row, head, to[m]);
        if (src < 0 || dst < 0) continue;
        const int64_t so = src * row_bytes + part * 16, d_o = dst * row_bytes + part * 16;
        *reinterpret_cast<u32x4_kv *>(c.k + d_o) = *reinterpret_cast<const u32x4_kv *>(c.k + so);
        *reinterpret_cast<u32x4_kv *>(c.v + d_o) = *reinterpret_cast<const u32x4_kv *>(c.v + so);
    }
}

int64_t kv_evict_workspace_bytes(const KvCache &c, int budget, int max_len) {
    if (max_len <= budget) return 0;
    const int64_t most = max_len - budget < budget ? max_len - budget : budget;
    return (int64_t)c.rows * c.heads * 2 * most * 4;
}

hipError_t launch_kv_evict(const KvCache &c, const KvEvict &a, hipStream_t stream) {
    hipLaunchKernelGGL(kv_evict_kernel, dim3((unsigned)c.rows * c.heads), dim3(EVICT_THREADS), 0, stream, c, a);
    return hipGetLastError();
}

}  // namespace nbw
