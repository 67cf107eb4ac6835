// paged_device.cuh -- device helpers of the paged-cache kernels and the rotary
// positions: exact rotary angles, typed loads and stores of 8 elements, and the
// Hadamard network of a row spread over 4 or 8 lanes.  Internal linkage: every
// translation unit gets its own copy.
#pragma once

#include "rot_device.cuh"

namespace rq {
namespace {

// cos and sin of position * frequency.  `turns` is the frequency in turns per
// position as a 64-bit binary fraction, so the wrapping product is the angle
// modulo one turn, exact for every position.  The nearest quarter turn is taken out of it
// in integers: what is left, an eighth of a turn at most either way, is off by 2^-28 turns
// (2.4e-8) at most as a float, where half a turn either way would be by 2^-26.
__device__ __forceinline__ float2 rotary_cos_sin(int64_t pos, uint64_t turns, float mscale) {
    const uint64_t phase = (uint64_t)pos * turns + (1ull << 61);
    const uint32_t quarter = (uint32_t)(phase >> 62);
    const int32_t rest = (int32_t)((uint32_t)(phase >> 30) ^ 0x80000000u);           // in 2^-34 turns
    float s, c;
    sincospif((float)rest * 1.1641532182693481e-10f, &s, &c);                        // 2^-33 half turns
    const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
    const float m = quarter & 2 ? -mscale : mscale;
    return make_float2(x * m, y * m);
}

template <int D>
__device__ __forceinline__ constexpr float inv_sqrt_dim() {
    return D == 32 ? 0.17677669529663687f : D == 64 ? 0.125f : D == 128 ? 0.08838834764831845f : 0.0625f;
}

// 8 consecutive elements (16 bytes, or 32 in fp32) at a 16-byte boundary, as 4 pairs.
template <int IN>
__device__ __forceinline__ void unpack8(const uint4 *r, pair_t *v) {
    if constexpr (IN == IN_F32) {
        const uint4 a = r[0], b = r[1];
        v[0] = ((pair_t)a.y << 32) | a.x;
        v[1] = ((pair_t)a.w << 32) | a.z;
        v[2] = ((pair_t)b.y << 32) | b.x;
        v[3] = ((pair_t)b.w << 32) | b.z;
    } else {
        const uint32_t w[4] = {r[0].x, r[0].y, r[0].z, r[0].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (IN == IN_BF16) {
                v[k] = ((pair_t)(w[k] & 0xffff0000u) << 32) | (pair_t)(w[k] << 16);
            } else {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
                v[k] = mk2(f.x, f.y);
            }
        }
    }
}
template <int IN>
__device__ __forceinline__ void load8(const void *p, pair_t (&v)[4]) {
    uint4 r[IN == IN_F32 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < (IN == IN_F32 ? 2 : 1); ++i) r[i] = static_cast<const uint4 *>(p)[i];
    unpack8<IN>(r, v);
}

// 4 pairs rounded to the element type (once, to nearest even).
template <int IN>
__device__ __forceinline__ void store8(void *p, const pair_t (&v)[4]) {
    if constexpr (IN == IN_F32) {
        static_cast<uint4 *>(p)[0] = make_uint4((uint32_t)v[0], (uint32_t)(v[0] >> 32), (uint32_t)v[1], (uint32_t)(v[1] >> 32));
        static_cast<uint4 *>(p)[1] = make_uint4((uint32_t)v[2], (uint32_t)(v[2] >> 32), (uint32_t)v[3], (uint32_t)(v[3] >> 32));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (IN == IN_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(lo2(v[k]), hi2(v[k]));
                w[k] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __half2 h = __floats2half2_rn(lo2(v[k]), hi2(v[k]));
                w[k] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        *static_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// 16 bytes as 8 (16-bit) or 4 (fp32) values, and back (rounded to nearest even).
template <int IN>
__device__ __forceinline__ void unpack16(const uint4 &x, float (&f)[IN == IN_F32 ? 4 : 8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (IN == IN_F32) {
            f[k] = __uint_as_float(w[k]);
        } else if constexpr (IN == IN_BF16) {
            f[2 * k] = __uint_as_float(w[k] << 16);
            f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
        } else {
            const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&w[k]));
            f[2 * k] = h.x;
            f[2 * k + 1] = h.y;
        }
    }
}
template <int IN>
__device__ __forceinline__ uint4 pack16(const float (&f)[IN == IN_F32 ? 4 : 8]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (IN == IN_F32) {
            w[k] = __float_as_uint(f[k]);
        } else if constexpr (IN == IN_BF16) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t *>(&h);
        } else {
            const __half2 h = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t *>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <int IN>
__device__ __forceinline__ void store_elem(void *base, int64_t i, float v) {
    if constexpr (IN == IN_F32) static_cast<float *>(base)[i] = v;
    else if constexpr (IN == IN_BF16) static_cast<__nv_bfloat16 *>(base)[i] = __float2bfloat16_rn(v);
    else static_cast<__half *>(base)[i] = __float2half_rn(v);
}

// A row of D elements over LPR lanes: lane l of the row holds the 8-element chunks
// l, l + LPR, l + 2 LPR, ... (so that each load instruction covers whole lines).
template <int D>
struct RowLanes {
    static constexpr int LPR = D == 256 ? 8 : 4;
    static constexpr int NCH = D / 8 / LPR;      // chunks per lane
    static constexpr int NP = 4 * NCH;           // pairs per lane
};

// Sylvester butterflies over all log2(D) index bits: in the pair, across the pairs
// of a chunk and the chunks of a lane in registers, across lanes by shuffles.
template <int D>
__device__ __forceinline__ void row_fwht(pair_t (&v)[RowLanes<D>::NP], int rl) {
    using L = RowLanes<D>;
#pragma unroll
    for (int i = 0; i < L::NP; ++i) v[i] = bfly_in(v[i]);
#pragma unroll
    for (int rb = 1; (1 << (rb - 1)) < L::NP; ++rb) butterfly_pairs(v, rb);
#pragma unroll
    for (int m = 1; m < L::LPR; m <<= 1) {
        const float sg = (rl & m) ? -1.f : 1.f;
        const pair_t sg2 = mk2(sg, sg);
#pragma unroll
        for (int i = 0; i < L::NP; ++i) v[i] = fma2(v[i], sg2, __shfl_xor_sync(0xffffffffu, v[i], m));
    }
}

// The row's sign vector as sign bits of this lane's elements (0 or 0x80000000 each).
template <int D>
__device__ __forceinline__ void row_sign_pairs(pair_t (&sg)[RowLanes<D>::NP], const uint32_t *sign_words, int rl) {
    using L = RowLanes<D>;
#pragma unroll
    for (int i = 0; i < L::NCH; ++i) {
        const int ch = rl + L::LPR * i;
        const uint32_t bits = sign_words[ch >> 2] >> (8 * (ch & 3));
#pragma unroll
        for (int k = 0; k < 4; ++k)
            sg[4 * i + k] = ((pair_t)((bits >> (2 * k + 1)) << 31) << 32) | (pair_t)(uint32_t)((bits >> (2 * k)) << 31);
    }
}
// sign_words[w] bit j: element 32 w + j is negated.  All threads of the block take
// part (D <= blockDim.x * 2, whole warps); followed by the caller's barrier.
template <int D>
__device__ __forceinline__ void block_sign_words(uint32_t *sign_words, uint64_t seed) {
    for (int e = threadIdx.x; e < D; e += blockDim.x) {
        const uint32_t w = __ballot_sync(0xffffffffu, (splitmix64_at(seed, (uint64_t)e) >> 63) != 0);
        if ((e & 31) == 0) sign_words[e >> 5] = w;
    }
}

// (x & mask) ^ flip in one instruction: two constants written out take two.
__device__ __forceinline__ uint32_t masked_flip(uint32_t x, uint32_t mask, uint32_t flip) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(y) : "r"(x), "r"(mask), "r"(flip));
    return y;
}

// A word of 8 codes as four pairs (nibbles j and j + 4) of fp16 codes, exactly.  0x6400 | u
// is 1024 + u, so nibbles 0 and 4 (u = code + 8 after the sign bit's flip) lose 1032;
// nibbles 1 and 5, which stay four bits up, are 1024 + 16 u: times 1/16, less 72.
__device__ __forceinline__ void code_pairs(uint32_t x, uint32_t (&r)[4]) {
    const __half2 m0 = __half2half2(__ushort_as_half(0xe408)), r16 = __half2half2(__ushort_as_half(0x2c00)),
                  m1 = __half2half2(__ushort_as_half(0xd480));             // -1032, 1/16, -72
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        const uint32_t y = x >> (4 * j);
        const uint32_t a = masked_flip(y, 0x000f000fu, 0x64086408u), b = masked_flip(y, 0x00f000f0u, 0x64806480u);
        const __half2 ha = __hadd2(*reinterpret_cast<const __half2 *>(&a), m0);
        const __half2 hb = __hfma2(*reinterpret_cast<const __half2 *>(&b), r16, m1);
        r[j] = *reinterpret_cast<const uint32_t *>(&ha);
        r[j + 1] = *reinterpret_cast<const uint32_t *>(&hb);
    }
}
}  // namespace
}  // namespace rq
