// kv_shared.hip -- attention of each row's new tokens over its cached slots, gfx950.
//
// One workgroup takes one token and query head: 256 slots at a time, a thread the score of one
// slot, then a thread the sum over the slots in one or more dims.  All arithmetic is fp32.
#include <algorithm>

#include "kv.h"

namespace nbw {

constexpr int SHARED_THREADS = 256;

template <bool FP8>
__device__ __forceinline__ float element(const uint8_t *row, int d) {
    if constexpr (FP8) return __builtin_amdgcn_cvt_f32_fp8(row[d], 0);
    else return __uint_as_float((uint32_t)((const uint16_t *)row)[d] << 16);
}

template <int DIM, bool FP8>
__global__ __launch_bounds__(SHARED_THREADS) void kv_shared_kernel(KvCache c, KvAttendShared a) {
    __shared__ float s_q[DIM], s_p[SHARED_THREADS], s_wave[SHARED_THREADS / 64];
    __shared__ int64_t s_at[SHARED_THREADS];
    const int tid = threadIdx.x, token = blockIdx.x / a.q_heads, qh = blockIdx.x % a.q_heads;
    const int head = qh / (a.q_heads / c.heads);
    int row = token, behind = 0;  // new tokens of the row after this one
    if (a.cu) {
        row = 0;
        for (int r = tid; r < (c.rows + SHARED_THREADS - 1) / SHARED_THREADS * SHARED_THREADS; r += SHARED_THREADS)
            row += __syncthreads_count(r < c.rows && a.cu[r + 1] <= token);
        if (row >= c.rows) return;
        behind = a.cu[row + 1] - 1 - token;
    }
    const int n = kv_len(a.lens, row, a.max_len) - behind;
    uint16_t *out = a.out + (int64_t)token * a.out_ld + (int64_t)qh * DIM;
    if (tid < DIM) s_q[tid] = __uint_as_float((uint32_t)a.q[(int64_t)token * a.q_ld + (int64_t)qh * DIM + tid] << 16);
    float m = -__builtin_inff(), sum = 0.f, o = 0.f;
    // The weights, up to 1 each, times a power of two sum to 1 at the most: finite values cannot run over.
    const float down = n > 1 ? __uint_as_float((uint32_t)(127 - (32 - __builtin_clz(n - 1))) << 23) : 1.f;
    constexpr int ROW = FP8 ? DIM : DIM * 2;
    const float by = a.scale * (FP8 ? c.k_scale[head] : 1.f);
    for (int j0 = 0; j0 < n; j0 += SHARED_THREADS) {
        __syncthreads();
        const int j = j0 + tid;
        const int64_t at = j < n ? kv_row(c, row, head, j) : -1;
        float s = -__builtin_inff();
        if (at >= 0) {
            s = 0.f;
            for (int d = 0; d < DIM; ++d) s += s_q[d] * element<FP8>(c.k + at * ROW, d);
            s *= by;
        }
        float top = s;
        for (int d = 1; d < 64; d <<= 1) {
            const float x = __shfl_xor(top, d);
            top = top >= x || top != top ? top : x;  // a NaN stays
        }
        if ((tid & 63) == 0) s_wave[tid >> 6] = top;
        __syncthreads();
        for (int w = 0; w < SHARED_THREADS / 64; ++w) top = top >= s_wave[w] || top != top ? top : s_wave[w];
        top = m >= top || m != m ? m : top;
        const float fade = m == top ? 1.f : expf(m - top);
        m = top;
        s_p[tid] = m == -__builtin_inff() ? 0.f : expf(s - m) * down;
        s_at[tid] = at;
        __syncthreads();
        sum *= fade;
        o *= fade;
        for (int i = 0; i < min(SHARED_THREADS, n - j0); ++i) {
            const int64_t row_at = s_at[i];
            if (row_at < 0) continue;
            sum += s_p[i];
            if (tid < DIM) o += s_p[i] * element<FP8>(c.v + row_at * ROW, tid);
        }
    }
    if (tid < DIM) out[tid] = to_bf16(m == -__builtin_inff() ? 0.f : o / sum * (FP8 ? c.v_scale[head] : 1.f));
}

int64_t kv_attend_shared_workspace_bytes(const KvCache &c, int q_heads, int tokens, int, int, int) {
    return fits_launch((int64_t)tokens * q_heads, SHARED_THREADS) ? 0 : -1;
}

hipError_t launch_kv_attend_shared(const KvCache &c, const KvAttendShared &a, int, hipStream_t stream) {
    const dim3 grid((unsigned)(a.tokens * a.q_heads)), threads(SHARED_THREADS);
#define NBW_SHARED(D, F) hipLaunchKernelGGL((kv_shared_kernel<D, F>), grid, threads, 0, stream, c, a)
    switch (c.dim) {
    case 64: if (c.fp8) NBW_SHARED(64, true); else NBW_SHARED(64, false); break;
    case 128: if (c.fp8) NBW_SHARED(128, true); else NBW_SHARED(128, false); break;
    default: if (c.fp8) NBW_SHARED(256, true); else NBW_SHARED(256, false); break;
    }
#undef NBW_SHARED
    return hipGetLastError();
}

}  // namespace nbw
