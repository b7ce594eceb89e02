// verify.hip -- which drafted tokens stand, and the token after them, gfx950.
//
// The drafts of a row are looked at side by side: a lane gathers p[x] and q[x] of
// one, and the first that is refused ends the row's run.  u q < p in fp64 is exact,
// the product of two numbers of 24 bits having 48.
//
// The next token is found in the running sum of one line's weights, max(p - q, 0) or p,
// which a first launch cuts into chunks of 4096 and sums, each chunk in a workgroup of
// its own whatever the rows; a second one, a workgroup for each row, finds the chunk
// that the sum passes u times the whole in, and then the place in it.  All sums
// are in fp64 and in a fixed order: of 128 thousand weights they are off by about
// 1e-14, so that the place is the exact one but for one draw in 1e9.
//
// Bound: memory, one line a row, or two where a draft was refused; for few rows the
// chain of loads (cu -> tokens -> p, q -> line) and the second launch.
#include <algorithm>

#include "kv.h"

namespace nbw {

constexpr int VERIFY_THREADS = 256;
constexpr int VERIFY_WAVES = VERIFY_THREADS / 64;
constexpr int EACH = 16;                        // weights of a thread
constexpr int SPAN = VERIFY_THREADS * EACH;     // weights of a chunk

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

// Eight bf16 or four fp32 numbers from an address that is only theirs to be aligned by.
template <bool BF16>
struct Pack {
    static constexpr int N = BF16 ? 8 : 4;
    u32x4_kv w;
    __device__ __forceinline__ void load(const void *p, int64_t i) {
        __builtin_memcpy(&w, (const uint8_t *)p + i * (BF16 ? 2 : 4), 16);
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (BF16) return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
        else return __uint_as_float(w[i]);
    }
};

// What a difference counts as a weight.
__device__ __forceinline__ double weight(double x) { return x > 0.0 && x < __builtin_inf() ? x : 0.0; }

// How many of a row's drafts stand; the same in all lanes of the wave that asks.
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

// The weights of elements [at, at + N) of a line, w, and what they are where no difference
// is above 0, p; elements past the vocabulary count as 0.
template <bool BF16>
struct Line {
    const void *target, *draft;  // draft: null if p alone counts
    int64_t p0, q0;              // the line's first element in each
    int vocab, out;              // the one token whose weight is 0 (-1: none)

    template <int N, class F>
    __device__ __forceinline__ void weights(int at, F use) const {
        if (at + N <= vocab) {
            Pack<BF16> p[N / Pack<BF16>::N], q[N / Pack<BF16>::N];
#pragma unroll
            for (int k = 0; k < N / Pack<BF16>::N; ++k) {
                p[k].load(target, p0 + at + k * Pack<BF16>::N);
                if (draft) q[k].load(draft, q0 + at + k * Pack<BF16>::N);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const double x = p[i / Pack<BF16>::N].get(i % Pack<BF16>::N);
                const double y = draft ? (double)q[i / Pack<BF16>::N].get(i % Pack<BF16>::N) : 0.0;
                use(i, at + i == out ? 0.0 : weight(x - y), weight(x));
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                double x = 0.0, y = 0.0;
                if (at + i < vocab) {
                    x = prob<BF16>(target, p0 + at + i);
                    if (draft) y = prob<BF16>(draft, q0 + at + i);
                }
                use(i, at + i == out ? 0.0 : weight(x - y), weight(x));
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

__device__ __forceinline__ double wave_sum64(double x) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d);
    return x;
}

// The first launch: the sums of each row's chunks, of the weights and of p.
template <bool BF16>
__global__ __launch_bounds__(VERIFY_THREADS) void verify_sums_kernel(VerifyDrafts a, int chunks, double *sums) {
    __shared__ double s_w[VERIFY_WAVES], s_p[VERIFY_WAVES];
    const int row = blockIdx.x / chunks, chunk = blockIdx.x % chunks, tid = threadIdx.x, wave = tid >> 6;
    const Lines l = lines_of(a, row);
    double w = 0.0, p = 0.0;
    if (l.count > 0) {
        const int stands = standing<BF16>(a, l);
        if (chunk == 0 && tid == 0) a.accepted[row] = stands;
        const Line<BF16> line = line_of<BF16>(a, l, stands);
        constexpr int N = Pack<BF16>::N;
#pragma unroll
        for (int k = 0; k < EACH / N; ++k) {
            // a wave's loads side by side
            const int64_t at = (int64_t)chunk * SPAN + k * (VERIFY_THREADS * N) + tid * N;
            if (at < a.vocab)
                line.template weights<N>((int)at, [&](int, double x, double y) {
                    w += x;
                    p += y;
                });
        }
    } else if (chunk == 0 && tid == 0) {
        a.accepted[row] = 0;
    }
    w = wave_sum64(w);
    p = wave_sum64(p);
    if ((tid & 63) == 0) {
        s_w[wave] = w;
        s_p[wave] = p;
    }
    __syncthreads();
    if (tid == 0) {
        for (int i = 1; i < VERIFY_WAVES; ++i) {
            w += s_w[i];
            p += s_p[i];
        }
        sums[2 * (int64_t)blockIdx.x] = w;
        sums[2 * (int64_t)blockIdx.x + 1] = p;
    }
}

// The sum of x over the workgroup's threads before this one, and over all.
struct Before {
    double mine, all;
};
__device__ __forceinline__ Before before_mine(double x, double *s_wave) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    double upto = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const double y = __shfl_up(upto, d);
        if (lane >= d) upto += y;
    }
    if (lane == 63) s_wave[wave] = upto;
    double mine = __shfl_up(upto, 1);
    if (lane == 0) mine = 0.0;
    __syncthreads();
    double lead = 0.0, all = 0.0;
    for (int w = 0; w < VERIFY_WAVES; ++w) {
        if (w < wave) lead += s_wave[w];
        all += s_wave[w];
    }
    __syncthreads();
    return {lead + mine, all};
}

// The second launch: each row's next token.
template <bool BF16>
__global__ __launch_bounds__(VERIFY_THREADS) void verify_next_kernel(VerifyDrafts a, int chunks, const double *sums) {
    __shared__ double s_wave[VERIFY_WAVES];
    __shared__ int s_first, s_last;
    __shared__ double s_before;
    const int row = blockIdx.x, tid = threadIdx.x;
    const Lines l = lines_of(a, row);
    if (l.count <= 0) {
        if (tid == 0) a.next[row] = -1;
        return;
    }
    Line<BF16> line = line_of<BF16>(a, l, a.accepted[row]);
    const double *mine = sums + 2 * (int64_t)row * chunks;
    if (tid == 0) {
        s_first = INT32_MAX;
        s_last = -1;
        s_before = 0.0;
    }
    // A thread has a run of chunks.
    const int run = (chunks + VERIFY_THREADS - 1) / VERIFY_THREADS, c0 = min(tid * run, chunks), c1 = min(c0 + run, chunks);
    double x = 0.0;
    for (int c = c0; c < c1; ++c) x += mine[2 * c];
    Before b = before_mine(x, s_wave);
    int of = 0;
    if (b.all == 0.0) {  // no difference above 0: p itself
        of = 1;
        line.draft = nullptr;
        line.out = -1;
        x = 0.0;
        for (int c = c0; c < c1; ++c) x += mine[2 * c + 1];
        b = before_mine(x, s_wave);
    }
    if (b.all == 0.0) {
        if (tid == 0) a.next[row] = -1;
        return;
    }
    const float u32 = a.u[l.first + l.count - 1];
    const double u = u32 > 0.f ? (u32 < 1.f ? (double)u32 : 1.0) : 0.0, goal = u * b.all;
    // The first chunk whose end is past the goal; should rounding leave none, the last that has any weight.
    double at = b.mine;
    for (int c = c0; c < c1; ++c) {
        const double own = mine[2 * c + of];
        if (own > 0.0) {
            atomicMax(&s_last, c);
            if (at + own > goal) {
                atomicMin(&s_first, c);
                break;
            }
        }
        at += own;
    }
    __syncthreads();
    const int chunk = s_first != INT32_MAX ? s_first : s_last;
    if (chunk >= c0 && chunk < c1) {
        at = b.mine;
        for (int c = c0; c < chunk; ++c) at += mine[2 * c + of];
        s_before = at;
    }
    __syncthreads();
    const double lead = s_before;
    if (tid == 0) {
        s_first = INT32_MAX;
        s_last = -1;
    }
    // The same in the chunk: a thread has EACH weights in a row.
    const int64_t first = (int64_t)chunk * SPAN + tid * EACH;
    double w[EACH];
    x = 0.0;
    if (first < a.vocab) {
        line.template weights<EACH>((int)first, [&](int i, double v, double) {
            w[i] = v;
            x += v;
        });
    } else {
#pragma unroll
        for (int i = 0; i < EACH; ++i) w[i] = 0.0;
    }
    b = before_mine(x, s_wave);
    if (x > 0.0) {
        at = lead + b.mine;
        int pick = -1, last = -1;
#pragma unroll
        for (int i = 0; i < EACH; ++i) {
            at += w[i];
            if (w[i] > 0.0) {
                last = i;
                if (pick < 0 && at > goal) pick = i;
            }
        }
        atomicMax(&s_last, (int)first + last);
        if (pick >= 0) atomicMin(&s_first, (int)first + pick);
    }
    __syncthreads();
    if (tid == 0) a.next[row] = s_first != INT32_MAX ? s_first : s_last;
}

static int chunks_of(int vocab) { return (int)(((int64_t)vocab + SPAN - 1) / SPAN); }

int64_t verify_drafts_workspace_bytes(int rows, int vocab) {
    if (!fits_launch((int64_t)rows * chunks_of(vocab), VERIFY_THREADS)) return -1;
    return (int64_t)rows * chunks_of(vocab) * 16;
}

hipError_t launch_verify_drafts(const VerifyDrafts &a, hipStream_t stream) {
    const int chunks = chunks_of(a.vocab);
    const dim3 grid((unsigned)((int64_t)a.rows * chunks)), rows((unsigned)a.rows), threads(VERIFY_THREADS);
    if (a.bf16) {
        hipLaunchKernelGGL(verify_sums_kernel<true>, grid, threads, 0, stream, a, chunks, (double *)a.ws);
        hipLaunchKernelGGL(verify_next_kernel<true>, rows, threads, 0, stream, a, chunks, (const double *)a.ws);
    } else {
        hipLaunchKernelGGL(verify_sums_kernel<false>, grid, threads, 0, stream, a, chunks, (double *)a.ws);
        hipLaunchKernelGGL(verify_next_kernel<false>, rows, threads, 0, stream, a, chunks, (const double *)a.ws);
    }
    return hipGetLastError();
}

}  // namespace nbw
