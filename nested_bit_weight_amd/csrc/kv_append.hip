// kv_append.hip -- new keys and values into the paged cache, gfx950.
//
// One workgroup takes one token: its q_heads + 2 * heads head vectors (queries
// to rotate, keys to rotate and store, values to store).  A head vector is the
// work of dim/16 lanes, each holding 8 elements of the first half and the 8
// elements that rotation pairs them with, so the pairs meet in one lane and the
// norm's sum of squares needs only log2(dim/16) shuffles.  A lane keeps its
// position's 8 cosines and sines in registers for all head vectors of the token.
//
// All arithmetic is fp32; a result is rounded once, when it is stored.
//
// Bound: memory.  15 thousand tokens of 48 head vectors of 128 (350 MB in and out):
// 66 us, 5.3 TB/s, above what a plain copy of 2 GiB reaches (4.9); 64 tokens, one for
// each row: 4 us, the chain of dependent loads (length, page number) and a launch.
#include "kv.h"

namespace nbw {

constexpr int APPEND_THREADS = 256;

template <int DIM, bool FP8>
__global__ __launch_bounds__(APPEND_THREADS) void kv_append_kernel(KvCache c, KvAppend a) {
    constexpr int L = DIM / 16;  // lanes of a head vector
    constexpr int HALF = DIM / 2;
    const int tid = threadIdx.x, token = blockIdx.x;
    if (token >= a.tokens) {  // the workgroups past the tokens': the rows' new lengths
        const int row = (token - a.tokens) * APPEND_THREADS + tid;
        if (row < c.rows) {
            const int64_t added = a.cu ? (int64_t)a.cu[row + 1] - a.cu[row] : 1;
            a.lens_out[row] = (int32_t)(kv_len(a.lens, row, c.cap) + added);
        }
        return;
    }
    // The token's row: the number of rows that end at or before it.
    int row = token, first = token;
    if (a.cu) {
        row = 0;
        for (int at = 0; at < c.rows; at += 64) {
            const int i = at + (tid & 63);
            const bool before = i < c.rows && a.cu[i + 1] <= token;
            row += __popcll(__ballot(before));
        }
        if (row >= c.rows) return;  // past the last row: cu does not reach the token
        first = a.cu[row];
    }
    const int64_t slot64 = (int64_t)kv_len(a.lens, row, c.cap) + (token - first);
    const bool fits = slot64 < c.cap && token >= first;
    const int slot = fits ? (int)slot64 : 0;
    const int32_t position = a.positions[token];
    const int lane = tid % L, unit = tid / L;

    float cs[8], sn[8];
    if (a.rope) {
        if (position >= 0 && position < a.rope_rows) {
            const float *t = a.rope + (int64_t)position * DIM + lane * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                cs[i] = t[i];
                sn[i] = t[HALF + i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) cs[i] = sn[i] = __builtin_nanf("");
        }
    }
    const int heads = a.q_heads + 2 * c.heads;
    for (int h0 = 0; h0 < heads; h0 += APPEND_THREADS / L) {
        const int h = h0 + unit;
        if (h >= heads) break;
        const bool is_q = h < a.q_heads, is_v = h >= a.q_heads + c.heads;
        const int hk = is_q ? h : is_v ? h - a.q_heads - c.heads : h - a.q_heads;
        const uint16_t *src = is_q ? a.q + (int64_t)token * a.q_ld
                              : is_v ? a.v + (int64_t)token * a.v_ld
                                     : a.k + (int64_t)token * a.k_ld;
        src += (int64_t)hk * DIM + lane * 8;
        const u32x4_kv lo = *reinterpret_cast<const u32x4_kv *>(src);
        const u32x4_kv hi = *reinterpret_cast<const u32x4_kv *>(src + HALF);
        float x[8], y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16_lo(lo[i]);
            x[2 * i + 1] = bf16_hi(lo[i]);
            y[2 * i] = bf16_lo(hi[i]);
            y[2 * i + 1] = bf16_hi(hi[i]);
        }
        const uint16_t *w = is_v ? nullptr : is_q ? a.q_norm : a.k_norm;
        if (w) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += x[i] * x[i] + y[i] * y[i];
#pragma unroll
            for (int d = 1; d < L; d <<= 1) sum += __shfl_xor(sum, d, L);
            const float by = 1.f / sqrtf(sum * (1.f / DIM) + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] *= by * __uint_as_float((uint32_t)w[lane * 8 + i] << 16);
                y[i] *= by * __uint_as_float((uint32_t)w[HALF + lane * 8 + i] << 16);
            }
        }
        if (a.rope && !is_v) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float p = x[i], q = y[i];
                x[i] = p * cs[i] - q * sn[i];
                y[i] = q * cs[i] + p * sn[i];
            }
        }
        if (!is_q && FP8) {
            const float s = is_v ? c.v_scale[hk] : c.k_scale[hk];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] /= s;
                y[i] /= s;
            }
        }
        if (!is_q) {
            const int64_t at = fits ? kv_row(c, row, hk, slot) : -1;
            if (at < 0) continue;
            uint8_t *pool = is_v ? c.v : c.k;
            if (FP8) {
                uint8_t *dst = pool + at * DIM + lane * 8;
                const u32x2_kv b0 = {to_fp8x4(x[0], x[1], x[2], x[3]), to_fp8x4(x[4], x[5], x[6], x[7])};
                const u32x2_kv b1 = {to_fp8x4(y[0], y[1], y[2], y[3]), to_fp8x4(y[4], y[5], y[6], y[7])};
                *reinterpret_cast<u32x2_kv *>(dst) = b0;
                *reinterpret_cast<u32x2_kv *>(dst + HALF) = b1;
                if (is_v || lane) continue;
            }
            if (!is_v && lane == 0) {
                const int64_t i = ((int64_t)row * c.heads + hk) * c.cap + slot;
                if (a.pos) a.pos[i] = position;
                if (a.acc) a.acc[i] = 0.f;
            }
            if (FP8) continue;
            u32x4_kv b0, b1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                b0[i] = to_bf16(x[2 * i]) | (uint32_t)to_bf16(x[2 * i + 1]) << 16;
                b1[i] = to_bf16(y[2 * i]) | (uint32_t)to_bf16(y[2 * i + 1]) << 16;
            }
            uint8_t *dst = pool + (at * DIM + lane * 8) * 2;
            *reinterpret_cast<u32x4_kv *>(dst) = b0;
            *reinterpret_cast<u32x4_kv *>(dst + HALF * 2) = b1;
        } else {
            u32x4_kv b0, b1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                b0[i] = to_bf16(x[2 * i]) | (uint32_t)to_bf16(x[2 * i + 1]) << 16;
                b1[i] = to_bf16(y[2 * i]) | (uint32_t)to_bf16(y[2 * i + 1]) << 16;
            }
            uint16_t *dst = a.q_out + (int64_t)token * a.q_out_ld + (int64_t)hk * DIM + lane * 8;
            *reinterpret_cast<u32x4_kv *>(dst) = b0;
            *reinterpret_cast<u32x4_kv *>(dst + HALF) = b1;
        }
    }
}

hipError_t launch_kv_append(const KvCache &c, const KvAppend &a, hipStream_t stream) {
    const int extra = a.lens_out ? (c.rows + APPEND_THREADS - 1) / APPEND_THREADS : 0;
    const dim3 grid((unsigned)a.tokens + extra);
    if (grid.x == 0) return hipSuccess;
#define NBW_APPEND(D, F)                                                                             \
    hipLaunchKernelGGL((kv_append_kernel<D, F>), grid, dim3(APPEND_THREADS), 0, stream, c, a)
    switch (c.dim) {
    case 64: if (c.fp8) NBW_APPEND(64, true); else NBW_APPEND(64, false); break;
    case 128: if (c.fp8) NBW_APPEND(128, true); else NBW_APPEND(128, false); break;
    default: if (c.fp8) NBW_APPEND(256, true); else NBW_APPEND(256, false); break;
    }
#undef NBW_APPEND
    return hipGetLastError();
}

}  // namespace nbw
