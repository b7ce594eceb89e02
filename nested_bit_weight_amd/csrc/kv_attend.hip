// kv_attend.hip -- attention of one new token for each row over its cached
// ones, gfx950.
//
// The plain kernel: one workgroup takes one (row, query head), puts the head's
// scores into the workspace, turns them into softmax weights there and adds up
// the values; a second kernel adds a key-value head's weights to the totals.
#include "kv.h"

namespace nbw {

constexpr int ATTEND_THREADS = 256;

template <bool FP8>
__device__ __forceinline__ float kv_at(const uint8_t *pool, int64_t i) {
    if (FP8) return fp8_at(pool[i], 0);
    return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(pool)[i] << 16);
}

template <int DIM, bool FP8>
__global__ __launch_bounds__(ATTEND_THREADS) void kv_attend_kernel(KvCache c, KvAttend a) {
    __shared__ float q[DIM];
    __shared__ float part[ATTEND_THREADS];
    const int tid = threadIdx.x;
    const int row = blockIdx.x / a.q_heads, g = blockIdx.x % a.q_heads;
    const int head = g / (a.q_heads / c.heads);
    const int n = kv_len(a.lens, row, a.max_len);
    float *p = reinterpret_cast<float *>(a.ws) + (int64_t)blockIdx.x * a.max_len;
    for (int d = tid; d < DIM; d += ATTEND_THREADS)
        q[d] = __uint_as_float((uint32_t)a.q[(int64_t)row * a.q_ld + (int64_t)g * DIM + d] << 16);
    __syncthreads();
    const float by = a.scale * (FP8 ? c.k_scale[head] : 1.f);
    float top = -__builtin_inff();
    for (int j = tid; j < n; j += ATTEND_THREADS) {
        const int64_t at = kv_row(c, row, head, j);
        float s = 0.f;
        if (at < 0) s = -__builtin_inff();
        else {
            for (int d = 0; d < DIM; ++d) s += q[d] * kv_at<FP8>(c.k, at * DIM + d);
            s *= by;
        }
        p[j] = s;
        top = fmaxf(top, s);
    }
    part[tid] = top;
    __syncthreads();
    for (int d = ATTEND_THREADS / 2; d; d >>= 1) {
        if (tid < d) part[tid] = fmaxf(part[tid], part[tid + d]);
        __syncthreads();
    }
    top = part[0] == -__builtin_inff() ? 0.f : part[0];
    __syncthreads();
    float sum = 0.f;
    for (int j = tid; j < n; j += ATTEND_THREADS) {
        const float e = expf(p[j] - top);
        p[j] = e;
        sum += e;
    }
    part[tid] = sum;
    __syncthreads();
    for (int d = ATTEND_THREADS / 2; d; d >>= 1) {
        if (tid < d) part[tid] += part[tid + d];
        __syncthreads();
    }
    const float inv = part[0] == 0.f ? 0.f : 1.f / part[0];
    __syncthreads();
    for (int j = tid; j < n; j += ATTEND_THREADS) p[j] *= inv;
    __syncthreads();
    for (int d0 = 0; d0 < DIM; d0 += 64) {
        const int d = d0 + (tid & 63);
        float o = 0.f;
        for (int j = tid >> 6; j < n; j += ATTEND_THREADS / 64) {
            const int64_t at = kv_row(c, row, head, j);
            if (at >= 0) o += p[j] * kv_at<FP8>(c.v, at * DIM + d);
        }
        part[tid] = o;
        __syncthreads();
        if (tid < 64) {
            o = 0.f;
            for (int w = 0; w < ATTEND_THREADS / 64; ++w) o += part[w * 64 + tid];
            a.out[(int64_t)row * a.out_ld + (int64_t)g * DIM + d] = to_bf16(FP8 ? o * c.v_scale[head] : o);
        }
        __syncthreads();
    }
}

__global__ __launch_bounds__(ATTEND_THREADS) void kv_totals_kernel(KvCache c, KvAttend a) {
    const int row = blockIdx.x / c.heads, head = blockIdx.x % c.heads, group = a.q_heads / c.heads;
    const int n = kv_len(a.lens, row, a.max_len);
    const float *p = reinterpret_cast<const float *>(a.ws) + ((int64_t)row * a.q_heads + head * group) * a.max_len;
    for (int j = threadIdx.x; j < n; j += ATTEND_THREADS) {
        float w = 0.f;
        for (int g = 0; g < group; ++g) w += p[(int64_t)g * a.max_len + j];
        const int64_t i = (int64_t)blockIdx.x * c.cap + j;
        a.acc_out[i] = a.decay * a.acc[i] + w;
    }
}

int64_t kv_attend_workspace_bytes(const KvCache &c, int q_heads, int max_len, bool, int) {
    return (int64_t)c.rows * q_heads * max_len * 4;
}

hipError_t launch_kv_attend(const KvCache &c, const KvAttend &a, int, hipStream_t stream) {
    const dim3 grid((unsigned)c.rows * a.q_heads);
#define NBW_ATTEND(D, F)                                                                             \
    hipLaunchKernelGGL((kv_attend_kernel<D, F>), grid, dim3(ATTEND_THREADS), 0, stream, c, a)
    switch (c.dim) {
    case 64: if (c.fp8) NBW_ATTEND(64, true); else NBW_ATTEND(64, false); break;
    case 128: if (c.fp8) NBW_ATTEND(128, true); else NBW_ATTEND(128, false); break;
    default: if (c.fp8) NBW_ATTEND(256, true); else NBW_ATTEND(256, false); break;
    }
#undef NBW_ATTEND
    if (a.acc)
        hipLaunchKernelGGL(kv_totals_kernel, dim3((unsigned)c.rows * c.heads), dim3(ATTEND_THREADS), 0, stream, c, a);
    return hipGetLastError();
}

}  // namespace nbw
