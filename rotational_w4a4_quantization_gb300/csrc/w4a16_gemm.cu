// w4a16_gemm.cu -- products of a few rows of activations with 4-bit weights (sm_103a).
//
//   y[m][c] = sum_g s[c][g] sum_{k in g} x[m][k] q[c][k]      (g: 128 codes, or the channel)
// x is not quantised: codes are exact in its 16-bit type, so the products are exact too, and
// fp32 rows go as three bf16 parts, 8 bits each.
//
// A block owns 16 channels and up to 64 rows; its warps split K in steps of 128 codes and meet
// in shared memory at the end.
//  * mma.sync m16n8k16, channels x rows.  A lane's 16 bytes of a channel's step are codes
//    32 c .. 32 c + 31 (c = lane % 4): words of 8 codes whose nibbles j and j + 4 are a pair of
//    operands.  The same permutation of k on the side of x drops out.
//  * a step's sum of 128 products begins from 0 in the tensor core (whose additions are not
//    rounded to nearest) and is scaled and added in fp32 outside.
#include "rq.h"
#include "rq_internal.h"
#include "paged_device.cuh"

namespace rq {
namespace {

constexpr int kGWarps = 8, kGThreads = 32 * kGWarps, kGChan = 16;

struct W16Params {
    const void *x;
    const uint8_t *w;
    const float *s;
    void *y;
    int64_t M, N, K, ldx;
    int out;                    // InType of y
    bool grouped;
};

template <int IN, bool FIRST>
__device__ __forceinline__ void mma_w16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (IN == IN_F16) {
        if constexpr (FIRST)
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                         : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                         : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
        else
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                         : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                         : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    } else {
        if constexpr (FIRST)
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                         : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                         : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
        else
            asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                         : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                         : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
}

// A word of 8 codes as four pairs (nibbles j and j + 4), exact.  bf16 has 7 bits behind the
// point: 0x4300 | u is 128 + u (u = code + 8), less 136.
template <int IN>
__device__ __forceinline__ void weight_pairs(uint32_t x, uint32_t (&r)[4]) {
    if constexpr (IN == IN_F16) {
        code_pairs(x, r);
    } else {
        const __nv_bfloat162 less = __bfloat162bfloat162(__ushort_as_bfloat16(0xc308));      // -136
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t u = ((x >> (4 * j)) & 0x000f000fu) ^ 0x43084308u;
            const __nv_bfloat162 h = __hadd2(*reinterpret_cast<const __nv_bfloat162 *>(&u), less);
            r[j] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
}

// The 8 elements of a row that go with a word of codes, as its pairs' other side: part h of
// (element j, element j + 4).
template <int IN, int PARTS>
__device__ __forceinline__ void row_pairs(const void *row, int64_t at, bool on, uint32_t (&b)[PARTS][4]) {
    if constexpr (IN == IN_F32) {
        float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
        if (on) {
            lo = *reinterpret_cast<const float4 *>(static_cast<const float *>(row) + at);
            hi = *reinterpret_cast<const float4 *>(static_cast<const float *>(row) + at + 4);
        }
        float a[4] = {lo.x, lo.y, lo.z, lo.w}, c[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int h = 0; h < PARTS; ++h) {
                // the upper half of a float is its first 8 bits; three of them are all 24
                const uint32_t u = __float_as_uint(a[j]), v = __float_as_uint(c[j]);
                b[h][j] = __byte_perm(u, v, 0x7632u);
                a[j] -= __uint_as_float(u & 0xffff0000u);
                c[j] -= __uint_as_float(v & 0xffff0000u);
            }
    } else {
        const uint4 v = on ? *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(row) + at) : make_uint4(0u, 0u, 0u, 0u);
        b[0][0] = __byte_perm(v.x, v.z, 0x5410u);
        b[0][1] = __byte_perm(v.x, v.z, 0x7632u);
        b[0][2] = __byte_perm(v.y, v.w, 0x5410u);
        b[0][3] = __byte_perm(v.y, v.w, 0x7632u);
    }
}

template <int IN, int MT>
__global__ void __launch_bounds__(kGThreads) w4a16_kernel(const __grid_constant__ W16Params p) {
    constexpr int PARTS = IN == IN_F32 ? 3 : 1;
    __shared__ float part[kGWarps][MT * 8][kGChan + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int64_t c0 = (int64_t)blockIdx.x * kGChan, m0 = (int64_t)blockIdx.y * MT * 8;
    const int64_t steps = p.K / 128, s0 = steps * warp / kGWarps, s1 = steps * (warp + 1) / kGWarps;
    const int64_t ch[2] = {min(c0 + g, p.N - 1), min(c0 + g + 8, p.N - 1)};     // past N: the last, never stored
    const uint8_t *const w0 = p.w + ch[0] * (p.K / 2) + 16 * c, *const w1 = p.w + ch[1] * (p.K / 2) + 16 * c;

    float sum[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[t][k] = 0.f;
    for (int64_t st = s0; st < s1; ++st) {
        const uint4 a0 = *reinterpret_cast<const uint4 *>(w0 + st * 64), a1 = *reinterpret_cast<const uint4 *>(w1 + st * 64);
        const float f0 = p.grouped ? p.s[ch[0] * steps + st] : 1.f, f1 = p.grouped ? p.s[ch[1] * steps + st] : 1.f;
        const uint32_t x0[4] = {a0.x, a0.y, a0.z, a0.w}, x1[4] = {a1.x, a1.y, a1.z, a1.w};
        float d[MT][4];
#pragma unroll
        for (int wd = 0; wd < 4; ++wd) {
            uint32_t q0[4], q1[4];
            weight_pairs<IN>(x0[wd], q0);
            weight_pairs<IN>(x1[wd], q1);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const int64_t m = m0 + 8 * t + g;
                uint32_t b[PARTS][4];
                row_pairs<IN, PARTS>(static_cast<const char *>(p.x) + (m < p.M ? m : 0) * p.ldx * (IN == IN_F32 ? 4 : 2),
                                     st * 128 + 32 * c + 8 * wd, m < p.M, b);
#pragma unroll
                for (int h = PARTS - 1; h >= 0; --h)                // small parts first
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t a[4] = {q0[2 * i], q1[2 * i], q0[2 * i + 1], q1[2 * i + 1]};
                        if (wd == 0 && i == 0 && h == PARTS - 1) mma_w16<IN, true>(d[t], a, b[h][2 * i], b[h][2 * i + 1]);
                        else mma_w16<IN, false>(d[t], a, b[h][2 * i], b[h][2 * i + 1]);
                    }
            }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            sum[t][0] = fmaf(d[t][0], f0, sum[t][0]);
            sum[t][1] = fmaf(d[t][1], f0, sum[t][1]);
            sum[t][2] = fmaf(d[t][2], f1, sum[t][2]);
            sum[t][3] = fmaf(d[t][3], f1, sum[t][3]);
        }
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) part[warp][8 * t + 2 * c + (k & 1)][g + 8 * (k >> 1)] = sum[t][k];
    __syncthreads();
    for (int i = threadIdx.x; i < MT * 8 * kGChan; i += kGThreads) {
        const int r = i / kGChan, cc = i % kGChan;
        const int64_t m = m0 + r, n = c0 + cc;
        if (m >= p.M || n >= p.N) continue;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kGWarps; ++w) v += part[w][r][cc];
        if (!p.grouped) v *= p.s[n];
        switch (p.out) {
            case IN_F32: store_elem<IN_F32>(p.y, m * p.N + n, v); break;
            case IN_BF16: store_elem<IN_BF16>(p.y, m * p.N + n, v); break;
            default: store_elem<IN_F16>(p.y, m * p.N + n, v);
        }
    }
}

template <int IN>
cudaError_t launch_w16(const W16Params &p, cudaStream_t stream) {
    const int mt = p.M <= 8 ? 1 : p.M <= 16 ? 2 : 4;
    const dim3 grid((unsigned)((p.N + kGChan - 1) / kGChan), (unsigned)((p.M + 8 * mt - 1) / (8 * mt)));
    if (mt == 1) w4a16_kernel<IN, 1><<<grid, kGThreads, 0, stream>>>(p);
    else if (mt == 2) w4a16_kernel<IN, 2><<<grid, kGThreads, 0, stream>>>(p);
    else w4a16_kernel<IN, 4><<<grid, kGThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_w4a16_gemm(const W16Call &c, cudaStream_t stream) {
    const W16Params p{c.x, c.w, c.scales, c.y, c.M, c.N, c.K, c.ldx, c.out_type, c.group != c.K};
    switch (c.in_type) {
        case IN_F32: return launch_w16<IN_F32>(p, stream);
        case IN_BF16: return launch_w16<IN_BF16>(p, stream);
        default: return launch_w16<IN_F16>(p, stream);
    }
}

}  // namespace rq
