// attn_tree_mma.cuh -- attention of trees of drafted tokens (or of single tokens) over
// the paged rotated INT4 cache (sm_103a): blocks of 8 or 16 query rows on mma.sync.
//
//   q~ = q R;  e_t = softmax_scale (q~ . k^_t) over the context and the visible
//   nodes;  p = softmax(e);  out = (sum_t p_t v^_t) R^T
// with k^_t = ks_t * codes, v^_t = vs_t * codes.  The G query heads of a KV head and
// the nodes of a sequence together are the rows of one product, so the cache is read
// once per block of rows.
//
//  * A block of 4 warps streams tiles of 128 tokens through a TMA ring; each warp
//    takes 32 of them (16 cost twice the waits, votes and query loads per token).  A
//    tile is codes of K and V (rows of D/2 bytes, swizzled by the TMA so that the reads
//    below are free of bank conflicts) and their scales.
//  * S = Q K^T: a lane reads the codes of a token straight into the B operand: nibbles j
//    and j + 4 of a word are a pair, and u = code + 8 in the low bits of an fp16 is the
//    subnormal u 2^-24 (16 u 2^-24 for odd j; q~ holds a sixteenth there): one logic
//    operation per pair and no arithmetic.  The row's factors take 2^24 and 8 sum q~ out
//    again, s = (a S + b) ks.  The order of the dims is the same permutation on both
//    sides and drops out.  fp32 queries subtract 8 from the codes instead: the offset
//    costs 5 bits of the sum.
//  * softmax on the fragments, base 2: a token's weight is w = 2^(s - z) vs, and a row's
//    reference z follows the row's own largest w, over the tokens that it sees: neither a
//    score whose values are nothing nor a value scale of no weight, or of another row's
//    tokens, costs the others bits.  It moves only when a weight passes 2^15, and then puts
//    it at 2^9: fp16 keeps 11 bits of weights down to 2^-14, so of tokens at least 23 bits
//    below the largest, and something down to 2^-25, and the accumulators are rarely
//    rescaled.  Whether one may is seen from the largest score and the largest scale of a
//    lane, and only then looked at token by token.
//  * O += w V: ldmatrix.trans pairs the codes of two tokens in a register, which is the B
//    operand after the same nibble step.  w is rounded to fp16 (11 bits, below the rounding
//    of 16-bit outputs); the sum of 2^(s - z) stays in fp32.
//  * Up to 8 rows (single tokens of up to 8 query heads to a KV head): the products are
//    turned, S^T = K q~^T and O^T = V^T P^T, with tokens and dims as the 16 of m16n8k16
//    and the rows as its 8.  The same registers are the operands, P^T passes through
//    movmatrix, and half of the products, of the softmax and of the accumulators is gone:
//    three blocks fit an SM (128 registers) where two did (168).
//  * fp32 queries: q~ and w are split into two fp16 parts and the products run twice; codes
//    are exact in either.  The second part of w is kept 2^11 up, so that small weights have
//    22 bits too.  What the tensor cores add to an accumulator is not rounded to nearest:
//    a score 17 to 26 bits above the others', added up by 16 of them, had its weight 5e-6
//    to 2e-5 off.  So each word of scores and each 16 tokens of outputs start from 0 and
//    are added to the sums outside, and the scale, with the rotation's 1/sqrt(D), has two
//    fp32 parts.  That and the second part's range cost 10 to 15% (18 sequences of 12k, 88
//    rows: 201 us for 179).  fp16 queries split q~
//    alone: their outputs resolve its rounding to 11 bits (4.6e-4 against 2.5e-4 of an
//    output).
//
// Measured (bf16, D = 128): 64 sequences of up to 8k, 8 query heads to each of 8 KV
// heads, one node: 83 us, 4.6 TB/s of cache, where 56 us is the reading alone (103 when a
// mask and a flip of codes took two instructions, and 130 then with blocks of 16 rows, half empty);
// two sequences of 256k, 4 query heads to a KV head: 106 us, 5.4 TB/s (135 and 167).  What bounds it is instructions (operands, softmax, fragments), so
// memory waits.  One sequence of 514 tokens takes the 16 us of its latencies and 7 of the
// join, which overlap in part.
#pragma once

#include "rq.h"
#include "rq_internal.h"
#include "tree_device.cuh"

namespace rq {
namespace {

constexpr int kTT = 128, kStages = 3, kCWarps = 4;
constexpr int kWT = kTT / kCWarps / 8;               // n8 tiles of tokens per warp and tile
constexpr int kMThreads = 32 * (kCWarps + 1);

// Blocks that share an SM: what the registers of the fragments allow.
constexpr int blocks_per_sm(int rows, int64_t head_dim) {
    return head_dim == 256 ? 1 : rows == 8 ? 3 : 2;
}

template <int IN, int D, int ROWS>
struct MSmem {
    static constexpr int RB = D / 2;
    static constexpr int HQ = IN == IN_BF16 ? 1 : 2, HP = IN == IN_F32 ? 2 : 1;   // fp16 parts of q~, of the weights
    alignas(1024) uint8_t kq[kStages][kTT * RB];
    alignas(1024) uint8_t vq[kStages][kTT * RB];
    alignas(16) float ks[kStages][kTT];
    alignas(16) float vs[kStages][kTT];
    alignas(16) uint32_t q[HQ][D / 16][32][ROWS / 4];  // q~ as fragments: k step, lane, register
    float acc[2][ROWS][D + 4];                       // the warps' sums, joined two by two
    float ref[kCWarps][ROWS], sum[kCWarps][ROWS];
    float2 rfac[ROWS];                               // a, b; fp32: a in two parts
    TreeLine line;
    alignas(8) uint64_t full[kStages], empty[kStages];
    uint32_t valid[kStages];
    volatile int abort_flag;
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// A word of 8 codes as code_pairs gives them, but as subnormals u 2^-24 and 16 u 2^-24,
// u = code + 8.
__device__ __forceinline__ void offset_pairs(uint32_t x, uint32_t (&r)[4]) {
    const uint32_t y = x >> 8;
    r[0] = masked_flip(x, 0x000f000fu, 0x00080008u);
    r[1] = masked_flip(x, 0x00f000f0u, 0x00800080u);
    r[2] = masked_flip(y, 0x000f000fu, 0x00080008u);
    r[3] = masked_flip(y, 0x00f000f0u, 0x00800080u);
}

// byte address of 16-byte chunk `ch` of row `row` in a tile written by TMA
template <int RB>
__device__ __forceinline__ uint32_t tile_chunk(int row, int ch) {
    if constexpr (RB == 128) ch ^= row & 7;
    else if constexpr (RB == 64) ch ^= (row >> 1) & 3;
    else if constexpr (RB == 32) ch ^= (row >> 2) & 1;
    return (uint32_t)(row * RB + ch * 16);
}

__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// The second part of fp32's weights is kept 2^11 larger, beside codes 2^-11 smaller (exact):
// what is left of a small weight would be subnormal.
constexpr float kLowUp = 2048.f;
__device__ __forceinline__ uint32_t lowered(uint32_t x) {
    const __half2 h = __hmul2(*reinterpret_cast<const __half2 *>(&x), __half2half2(__ushort_as_half(0x1000)));   // 2^-11
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ void add4(float (&to)[4], const float (&x)[4]) {
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
        const float2 y = __fadd2_rn(make_float2(to[k], to[k + 1]), make_float2(x[k], x[k + 1]));
        to[k] = y.x;
        to[k + 1] = y.y;
    }
}
// An 8 x 8 matrix of fp16 pairs, transposed across the warp.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ float2 unpack_h2(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2 *>(&x)); }

template <int IN, int D, int ROWS, class P>
__global__ void __launch_bounds__(kMThreads, blocks_per_sm(ROWS, D))
attn_tree_mma_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                     const __grid_constant__ P p) {
    using S = MSmem<IN, D, ROWS>;
    constexpr int RB = D / 2, WPT = D / 32, E = D / 32, HQ = S::HQ, HP = S::HP;
    constexpr bool kOffset = IN != IN_F32;             // keys as u = code + 8 (see the top)
    constexpr bool kShort = IN == IN_F32;              // the tensor cores add up few products, the rest is added outside
    constexpr int NQ = D / 32;                        // 16-byte chunks of a code row
    constexpr bool SIDE = ROWS == 8;                  // products of tokens x rows instead of rows x tokens
    constexpr int kRowLo = SIDE ? 4 : 1, kRowHi = SIDE ? 32 : 4;   // lane bits that a row's scores are spread over
    extern __shared__ uint8_t raw[];
    S &s = *reinterpret_cast<S *>(raw + ((1024u - (t_smem(raw) & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            t_mbar_init(&s.full[i], 1);
            t_mbar_init(&s.empty[i], kCWarps);
        }
        s.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tree_join_may_begin();
    tree_scan<ROWS, kTT>(p, s.line);               // ends with a block barrier
    if constexpr (P::kPass) {
        if (p.out_pass) tree_clear<ROWS, kTT>(p);
    }
    const int64_t total = s.line.prefix[kScan];
    const int64_t begin = tree_begin(total, p.ctas, blockIdx.x), end = tree_begin(total, p.ctas, blockIdx.x + 1);
    if constexpr (P::kPass) {
        if (begin == end) tree_empty<ROWS, D>(p);
    }
    int st = 0;
    uint32_t ph = 0;

    if (warp == kCWarps) {
        // ---------------- producer: one lane per page piece of a tile ----------------
        const int bt = min(kTT, 1 << p.log_page), pieces = kTT / bt;
        TreeJoin join{};
        for (int64_t at = begin; at < end;) {
            const TreeWork w = tree_work<ROWS, kTT>(p, s.line, at, begin, end);
            at += w.used;
            if (w.t1 <= w.t0) continue;
            auto page_of = [&](int tile) -> int64_t {
                const int t = tile * kTT + lane * bt;
                if (lane >= pieces || t >= w.s.len) return -1;
                const int64_t pg = p.table[w.b * p.width + (t >> p.log_page)];
                return pg >= 0 && pg < p.pages ? pg : -1;
            };
            int64_t pg = page_of(w.t0);
            for (int tile = w.t0; tile < w.t1; ++tile) {
                const int64_t next = tile + 1 < w.t1 ? page_of(tile + 1) : -1;
                const bool go = t_mbar_wait<P::kPass>(&s.empty[st], ph ^ 1, &s.abort_flag, p.err);
                const uint32_t valid = __ballot_sync(0xffffffffu, pg >= 0 && go);
                if (lane == 0) {
                    s.valid[st] = valid;
                    t_mbar_expect(&s.full[st], __popc(valid) * bt * (2 * RB + 8));
                }
                __syncwarp();
                if ((valid >> lane) & 1) {
                    const int t = tile * kTT + lane * bt;
                    const int64_t row = ((pg * p.kv_heads + w.h) << p.log_page) + (t & ((1 << p.log_page) - 1));
                    t_tma_2d(s.kq[st] + lane * bt * RB, &tmk, &s.full[st], (int)row);
                    t_bulk(&s.ks[st][lane * bt], p.ks + row, bt * 4, &s.full[st]);
                    t_tma_2d(s.vq[st] + lane * bt * RB, &tmv, &s.full[st], (int)row);
                    t_bulk(&s.vs[st][lane * bt], p.vs + row, bt * 4, &s.full[st]);
                }
                pg = next;
                if (++st == kStages) {
                    st = 0;
                    ph ^= 1;
                }
            }
            if constexpr (P::kPass) {
                if (p.out_pass && p.place) {
                    tree_place<ROWS>(p, s.line, w, begin, end);
                    continue;
                }
            }
            tree_note<ROWS, D>(p, s.line, w, begin, end, join);
        }
        tree_noted<ROWS, D>(p, join);
        if constexpr (P::kPass) pass_wait();
        // no copy outlives the block, also when it gave up
        if (s.abort_flag) {
            const long long t0 = clock64();
            while (clock64() - t0 < 20000000ll) __nanosleep(1000);
        }
        return;
    }

    // ---------------- consumers ----------------
    const int g = lane >> 2, c = lane & 3;
    auto cta_sync = [] { asm volatile("bar.sync 1, 128;" ::: "memory"); };
    float sg[E];
    lane_signs<E>(sg, lane, p.seed);
    const bool signs_first = (p.flags & RQ_SIGNS_FIRST) != 0;

    for (int64_t at = begin; at < end;) {
        const TreeWork w = tree_work<ROWS, kTT>(p, s.line, at, begin, end);
        at += w.used;
        if (w.t1 <= w.t0) continue;
        const int rows = min(ROWS, w.s.n * p.group - w.mt * ROWS);

        // ---- q~ of the block's rows: rotated in fp32, scaled by a power of two to below
        // 1 (its inverse goes into the row's score factor), rounded to fp16 once ----
        constexpr int RW = ROWS / kCWarps;                  // rows warp, warp + 4, ... : all at once
        float qv[RW][E];
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int r = i * kCWarps + warp, gr = w.mt * ROWS + r;
            const char *src = static_cast<const char *>(p.q) +
                              ((w.s.row0 + gr / p.group) * p.q_token + (w.h * p.group + gr % p.group) * p.q_head) *
                                  (IN == IN_F32 ? 4 : 2);
#pragma unroll
            for (int e = 0; e < E; ++e) qv[i][e] = r < rows ? load_elem<IN>(src, lane * E + e) : 0.f;
        }
        float top[RW], qsum[RW];
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            warp_rotate<E>(qv[i], sg, lane, signs_first, kOffset ? inv_sqrt_dim<D>() : 1.f);
            top[i] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) top[i] = fmaxf(top[i], fabsf(qv[i][e]));
        }
#pragma unroll
        for (int o = 16; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < RW; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int r = i * kCWarps + warp;
            // 2^ex > top, within what a float's exponent holds
            const int ex = max(-100, min((int)((__float_as_uint(top[i]) >> 23) & 255u) - 126, 100));
            const float down = __uint_as_float((uint32_t)(127 - ex) << 23), up = __uint_as_float((uint32_t)(127 + ex) << 23);
            top[i] = kOffset ? up * p.score_scale : up;
            qsum[i] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) {
                // lane column c of the fragments covers words of 8 dims: those of the 16-byte
                // chunk(s) of a code row that its K operand comes from
                const int d = lane * E + e, j = d & 3;
                const int fc = D == 256 ? (d >> 5) & 3 : d / (D / 4), wd = D == 256 ? ((d >> 7) << 2) + ((d & 31) >> 3) : (d % (D / 4)) >> 3;
                const int reg = SIDE ? j & 1 : (j & 1) * 2 + (r >> 3);
                const int at_q = (((2 * wd + (j >> 1)) * 32 + (r & 7) * 4 + fc) * (ROWS / 4) + reg) * 2 + ((d >> 2) & 1);
                const float x = qv[i][e] * (kOffset && (d & 1) ? 0.0625f * down : down);
                const __half hi = __float2half_rn(x);
                float got = __half2float(hi);
                reinterpret_cast<__half *>(s.q[0])[at_q] = hi;
                if constexpr (HQ == 2) {
                    const __half lo = __float2half_rn(x - got);
                    reinterpret_cast<__half *>(s.q[1])[at_q] = lo;
                    got += __half2float(lo);
                }
                qsum[i] += d & 1 ? 16.f * got : got;
            }
        }
        if constexpr (kOffset) {
#pragma unroll
            for (int o = 16; o; o >>= 1)
#pragma unroll
                for (int i = 0; i < RW; ++i) qsum[i] += __shfl_xor_sync(0xffffffffu, qsum[i], o);
        }
        if (lane == 0) {
#pragma unroll
            for (int i = 0; i < RW; ++i)
                s.rfac[i * kCWarps + warp] = kOffset ? make_float2(top[i] * 16777216.f, -8.f * qsum[i] * top[i])
                                                               : make_float2(top[i] * p.full_scale.x, top[i] * p.full_scale.y);
        }
        cta_sync();

        // this lane's two rows of scores
        const int row0 = SIDE ? 2 * c : g, row1 = SIDE ? 2 * c + 1 : g + 8;
        const float2 rs0 = s.rfac[row0], rs1 = s.rfac[row1];

        constexpr int NA = SIDE ? NQ * 2 : NQ * 4;
        float acc[NA][4];
#pragma unroll
        for (int i = 0; i < NA; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) acc[i][k] = 0.f;
        float z0 = 0.f, z1 = 0.f, l0 = 0.f, l1 = 0.f;                                     // references, sums
        float lim0 = -INFINITY, lim1 = -INFINITY;                                         // a weight beyond moves the reference

        const uint32_t all = (uint32_t)((1ull << (kTT / min(kTT, 1 << p.log_page))) - 1);
        for (int tile = w.t0; tile < w.t1; ++tile) {
            const bool ok = __all_sync(0xffffffffu, t_mbar_wait<false>(&s.full[st], ph, &s.abort_flag, p.err));
            const int tk = warp * 8 * kWT;                            // this warp's tokens of the tile
            const int t_first = tile * kTT + tk;
            if (ok && t_first < w.s.len) {
                // ---- S = Q K^T ----
                constexpr int NS = SIDE ? kWT / 2 : kWT;
                float sc[NS][4];
                constexpr int KP = WPT < 4 ? WPT : 4;                 // words loaded at once
                const uint8_t *krow = s.kq[st] + (tk + g) * RB;
#pragma unroll
                for (int part = 0; part < WPT / KP; ++part) {
                    uint32_t kw[kWT][KP];
#pragma unroll
                    for (int t = 0; t < kWT; ++t) {
                        // rows 8 apart have the same swizzle
                        if constexpr (D == 32) {
                            kw[t][0] = *reinterpret_cast<const uint32_t *>(krow + t * 8 * RB + 4 * c);
                        } else if constexpr (D == 64) {
                            const uint2 x = *reinterpret_cast<const uint2 *>(krow + t * 8 * RB + tile_chunk<RB>(g, c >> 1) - g * RB + 8 * (c & 1));
                            kw[t][0] = x.x; kw[t][1] = x.y;
                        } else {
                            const uint4 x = *reinterpret_cast<const uint4 *>(krow + t * 8 * RB + tile_chunk<RB>(g, c + 4 * part) - g * RB);
                            kw[t][0] = x.x; kw[t][1] = x.y; kw[t][2] = x.z; kw[t][3] = x.w;
                        }
                    }
#pragma unroll
                    for (int wd = 0; wd < KP; ++wd) {
                        uint32_t b[kWT][4];
#pragma unroll
                        for (int t = 0; t < kWT; ++t) {
                            if constexpr (kOffset) offset_pairs(kw[t][wd], b[t]);
                            else code_pairs(kw[t][wd], b[t]);
                        }
                        float own[kShort ? NS : 1][4];                  // this word's sums (kShort)
#pragma unroll
                        for (int step = 0; step < 2 * HQ; ++step) {
                            // kShort: the small part first, so that fewer additions meet the large one
                            const int hv = kShort ? HQ - 1 - step / 2 : step / 2, i = step & 1;
                            const bool begins = step == 0 && (kShort || (part == 0 && wd == 0));
                            auto add = [&](int t, const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
                                float(&to)[4] = kShort ? own[t % (kShort ? NS : 1)] : sc[t];
                                if (begins) mma16816_first(to, a, b0, b1);
                                else mma16816(to, a, b0, b1);
                            };
                            if constexpr (SIDE) {
                                const uint2 x = *reinterpret_cast<const uint2 *>(s.q[hv][2 * (part * KP + wd) + i][lane]);
#pragma unroll
                                for (int t = 0; t < NS; ++t) {
                                    const uint32_t a[4] = {b[2 * t][2 * i], b[2 * t + 1][2 * i], b[2 * t][2 * i + 1], b[2 * t + 1][2 * i + 1]};
                                    add(t, a, x.x, x.y);
                                }
                            } else {
                                const uint4 x = *reinterpret_cast<const uint4 *>(s.q[hv][2 * (part * KP + wd) + i][lane]);
                                const uint32_t a[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                for (int t = 0; t < kWT; ++t) add(t, a, b[t][2 * i], b[t][2 * i + 1]);
                            }
                        }
                        if constexpr (kShort) {
#pragma unroll
                            for (int t = 0; t < NS; ++t) {
                                if (part == 0 && wd == 0) {
#pragma unroll
                                    for (int k = 0; k < 4; ++k) sc[t][k] = own[t][k];
                                } else {
                                    add4(sc[t], own[t]);
                                }
                            }
                        }
                    }
                }
                // ---- scores against the references: s - z ----
                // sc[t][k]: row k < 2 of the lane's two where rows lead, k & 1 where tokens do;
                // token tok(t, k) of the warp's
                float2 vscale[NS];
                const float *ks = s.ks[st] + tk + (SIDE ? g : 2 * c), *vs = s.vs[st] + tk + (SIDE ? g : 2 * c);
                auto second = [](int k) { return SIDE ? (k & 1) != 0 : k >= 2; };          // of the two rows
                auto later = [](int k) { return SIDE ? k >= 2 : (k & 1) != 0; };           // of the two tokens
                auto tok = [&](int t, int k) { return SIDE ? 16 * t + 8 * (k >> 1) + g : 8 * t + 2 * c + (k & 1); };
#pragma unroll
                for (int t = 0; t < NS; ++t) {
                    float2 kk;
                    if constexpr (SIDE) {
                        kk = make_float2(ks[16 * t], ks[16 * t + 8]);
                        vscale[t] = make_float2(vs[16 * t], vs[16 * t + 8]);
                    } else {
                        kk = *reinterpret_cast<const float2 *>(ks + 8 * t);
                        vscale[t] = *reinterpret_cast<const float2 *>(vs + 8 * t);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 rs = second(k) ? rs1 : rs0;
                        sc[t][k] = fmaf(fmaf(sc[t][k], rs.x, kOffset ? rs.y : sc[t][k] * rs.y), later(k) ? kk.y : kk.x, second(k) ? -z1 : -z0);
                    }
                }
                const uint32_t valid = s.valid[st];
                const bool masked = t_first + 8 * kWT > w.s.ctx || valid != all;
                if (masked) {
                    const int lp = min(p.log_page, 7);
#pragma unroll
                    for (int t = 0; t < NS; ++t) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int tl = tk + tok(t, k);
                            const bool sees = ((valid >> (tl >> lp)) & 1) &&
                                              tree_sees<ROWS>(p, w, second(k) ? row1 : row0, tile * kTT + tl);
                            if (!sees) sc[t][k] = -INFINITY;
                        }
                    }
                }
                // ---- lazy references ----
                // largest score and largest value scale of the lane together bound its weights
                float up0 = -INFINITY, up1 = -INFINITY, vtop = 0.f;
#pragma unroll
                for (int t = 0; t < NS; ++t) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float &up = second(k) ? up1 : up0;
                        up = fmaxf(up, sc[t][k]);
                    }
                    vtop = fmaxf(vtop, fmaxf(vscale[t].x, vscale[t].y));
                }
                const float lv = fmaxf((float)((int)(__float_as_uint(vtop) >> 23) - 126), kLeastValue);
                if (__any_sync(0xffffffffu, up0 + lv > lim0 || up1 + lv > lim1)) {
                    // the rows' largest weights: a row's own, over the tokens that it sees
                    float w0 = -INFINITY, w1 = -INFINITY;
#pragma unroll
                    for (int t = 0; t < NS; ++t) {
                        const float lx = fmaxf(lg2(vscale[t].x), kLeastValue), ly = fmaxf(lg2(vscale[t].y), kLeastValue);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float &w = second(k) ? w1 : w0;
                            w = fmaxf(w, sc[t][k] + fminf(later(k) ? ly : lx, 128.f));
                        }
                    }
#pragma unroll
                    for (int o = kRowLo; o < kRowHi; o <<= 1) {
                        w0 = fmaxf(w0, __shfl_xor_sync(0xffffffffu, w0, o));
                        w1 = fmaxf(w1, __shfl_xor_sync(0xffffffffu, w1, o));
                    }
                    // z is 0 until something is seen (lim = -inf: the first weight moves it)
                    const float d0 = w0 > lim0 ? w0 - kWeightTo : 0.f, d1 = w1 > lim1 ? w1 - kWeightTo : 0.f;
                    const float f0 = lim0 == kWeightMost ? ex2(-d0) : 1.f, f1 = lim1 == kWeightMost ? ex2(-d1) : 1.f;
                    if (w0 != -INFINITY) lim0 = kWeightMost;
                    if (w1 != -INFINITY) lim1 = kWeightMost;
                    z0 += d0; z1 += d1;
                    l0 *= f0; l1 *= f1;
#pragma unroll
                    for (int t = 0; t < NS; ++t)
#pragma unroll
                        for (int k = 0; k < 4; ++k) sc[t][k] -= second(k) ? d1 : d0;
#pragma unroll
                    for (int i = 0; i < NA; ++i)
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[i][k] *= second(k) ? f1 : f0;
                }
                // ---- weights ----
#pragma unroll
                for (int t = 0; t < NS; ++t) {
                    bool hidden[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        hidden[k] = masked && sc[t][k] == -INFINITY;
                        sc[t][k] = ex2(sc[t][k]);
                    }
                    l0 += SIDE ? sc[t][0] + sc[t][2] : sc[t][0] + sc[t][1];
                    l1 += SIDE ? sc[t][1] + sc[t][3] : sc[t][2] + sc[t][3];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        sc[t][k] *= later(k) ? vscale[t].y : vscale[t].x;
                        if (masked && hidden[k]) sc[t][k] = 0.f;   // also where the value's scale is not finite
                    }
                }
                // ---- O += (P vs) V, 16 tokens at a time ----
                const uint32_t vbase = t_smem(s.vq[st]);
                const int mrow = tk + ((lane >> 3) & 1) * 8 + (lane & 7);
#pragma unroll
                for (int h = 0; h < kWT / 2; ++h) {
                    uint32_t pa[HP][4];                             // SIDE: two registers of each
                    if constexpr (SIDE) {
                        // [token][row] -> [row][token]
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const float *x = sc[h] + 2 * t;
                            const uint32_t hi = pack_h2(x[0], x[1]);
                            pa[0][t] = transposed(hi);
                            if constexpr (HP == 2) {
                                const float2 a = unpack_h2(hi);
                                pa[1][t] = transposed(pack_h2((x[0] - a.x) * kLowUp, (x[1] - a.y) * kLowUp));
                            }
                        }
                    } else {
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const float *x = sc[(2 * h + t) % NS];
                            pa[0][2 * t] = pack_h2(x[0], x[1]);
                            pa[0][2 * t + 1] = pack_h2(x[2], x[3]);
                            if constexpr (HP == 2) {
                                const float2 a = unpack_h2(pa[0][2 * t]), b = unpack_h2(pa[0][2 * t + 1]);
                                pa[1][2 * t] = pack_h2((x[0] - a.x) * kLowUp, (x[1] - a.y) * kLowUp);
                                pa[1][2 * t + 1] = pack_h2((x[2] - b.x) * kLowUp, (x[3] - b.y) * kLowUp);
                            }
                        }
                    }
                    auto pv = [&](int q, uint32_t x, uint32_t y) {
                        uint32_t b0[4], b1[4];
                        code_pairs(x, b0);
                        code_pairs(y, b1);
                        // a product of 16 tokens; kShort: both parts from 0, then added to the sums
                        auto product = [&](float(&to)[4], auto part) {
                            if constexpr (kShort) {
                                float own[4];
                                part(0, [&](const uint32_t (&a)[4], uint32_t x0, uint32_t x1) { mma16816_first(own, a, x0, x1); });
                                part(1, [&](const uint32_t (&a)[4], uint32_t x0, uint32_t x1) { mma16816(own, a, x0, x1); });
                                add4(to, own);
                            } else {
                                part(0, [&](const uint32_t (&a)[4], uint32_t x0, uint32_t x1) { mma16816(to, a, x0, x1); });
                            }
                        };
                        if constexpr (SIDE) {
#pragma unroll
                            for (int j = 0; j < 4; j += 2)
                                product(acc[2 * q + j / 2], [&](int hv, auto run) {
                                    const uint32_t a[4] = {hv ? lowered(b0[j]) : b0[j], hv ? lowered(b0[j + 1]) : b0[j + 1],
                                                           hv ? lowered(b1[j]) : b1[j], hv ? lowered(b1[j + 1]) : b1[j + 1]};
                                    run(a, pa[hv % HP][0], pa[hv % HP][1]);
                                });
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                product(acc[(4 * q + j) % NA], [&](int hv, auto run) {
                                    run(pa[hv % HP], hv ? lowered(b0[j]) : b0[j], hv ? lowered(b1[j]) : b1[j]);
                                });
                        }
                    };
                    if constexpr (NQ == 1) {
                        uint32_t x, y;
                        asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
                                     : "=r"(x), "=r"(y) : "r"(vbase + tile_chunk<RB>(mrow + 16 * h, 0)) : "memory");
                        pv(0, x, y);
                    } else {
#pragma unroll
                        for (int q = 0; q < NQ; q += 2) {
                            uint32_t x[4];
                            asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                                         : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                                         : "r"(vbase + tile_chunk<RB>(mrow + 16 * h, q + (lane >> 4))) : "memory");
                            pv(q, x[0], x[1]);
                            pv(q + 1, x[2], x[3]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) t_mbar_arrive(&s.empty[st]);
            if (++st == kStages) {
                st = 0;
                ph ^= 1;
            }
        }

        // ---- join the warps: references first, then the sums two by two ----
#pragma unroll
        for (int o = kRowLo; o < kRowHi; o <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, o);
            l1 += __shfl_xor_sync(0xffffffffu, l1, o);
        }
        const float m0 = lim0 == kWeightMost || !(l0 == 0.f) ? z0 : -INFINITY, m1 = lim1 == kWeightMost || !(l1 == 0.f) ? z1 : -INFINITY;
        if (SIDE ? g == 0 : c == 0) {
            s.ref[warp][row0] = m0;
            s.ref[warp][row1] = m1;
            s.sum[warp][row0] = l0;
            s.sum[warp][row1] = l1;
        }
        cta_sync();
        auto joined = [&](int r, float &top, float &sum) {
            top = -INFINITY;
#pragma unroll
            for (int i = 0; i < kCWarps; ++i) top = fmaxf(top, s.ref[i][r]);
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < kCWarps; ++i)
                if (s.ref[i][r] != -INFINITY) sum += s.sum[i][r] * ex2(s.ref[i][r] - top);
        };
        float top0, top1, sum0, sum1;
        joined(row0, top0, sum0);
        joined(row1, top1, sum1);
        const float f0 = m0 == -INFINITY ? 0.f : ex2(m0 - top0), f1 = m1 == -INFINITY ? 0.f : ex2(m1 - top1);
        // accumulators: dims 32 q + 8 c + j and + 4 + j of rows g, g + 8; SIDE: dim 32 q + 4 g + j
        // of rows 2 c, 2 c + 1
#pragma unroll
        for (int step = 0; step < 2; ++step) {
            if ((warp >> 1) == 1 - step) {                  // warps 2, 3 write, then 0, 1 add
                float(*dst)[D + 4] = s.acc[warp & 1];
#pragma unroll
                for (int q = 0; q < NQ; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int k = 0; k < 2; ++k)
#pragma unroll
                            for (int u = 0; u < (SIDE ? 1 : 2); ++u) {
                                // row k of the lane's two; u: the second of its dims
                                const float f = k ? f1 : f0;
                                const float a = SIDE ? acc[(2 * q + j / 2) % NA][2 * (j & 1) + k] : acc[(4 * q + j) % NA][2 * k + u];
                                float *x = &dst[k ? row1 : row0][32 * q + (SIDE ? 4 * g : 8 * c + 4 * u) + j];
                                const float val = f == 0.f ? 0.f : a * f;
                                *x = step == 0 ? val : *x + val;
                            }
            }
            cta_sync();
        }
        // ---- rows out: finished, or as a partial ----
        float *part = p.part, *ml = p.part + (int64_t)2 * p.ctas * ROWS * D;
        const int64_t slot = tree_slot(w, begin);
        float vsum[RW];
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int r = i * kCWarps + warp;
            joined(r, top[i], vsum[i]);
#pragma unroll
            for (int e = 0; e < E; ++e) qv[i][e] = s.acc[0][r][lane * E + e] + s.acc[1][r][lane * E + e];
        }
        const bool resumes = P::kPass && !out_pass(p) && w.begins && w.t0 == 0;       // from the pass before
        if constexpr (P::kPass) {
            if (resumes) pass_wait();
        }
        if (!w.begins || resumes) {                         // the pieces before this one
            // 16 rows, and rows of a pass: rolled, as short calls take their time fetching code
#pragma unroll(SIDE && !P::kPass ? RW : 1)
            for (int i = 0; i < RW; ++i) {
                const int r = i * kCWarps + warp;
                const float2 *const from_ml = reinterpret_cast<const float2 *>(ml + (slot * ROWS + r) * 2);
                const float *const from = part + (slot * ROWS + r) * D + lane * E;
                if constexpr (P::kPass) {
                    if (r >= rows) continue;
                    const TreeBefore before = resumes ? tree_before<D>(p, tree_state<ROWS>(p, w.s.row0, w.mt, w.h, r))
                                                      : TreeBefore{from_ml, from_ml, from, from, 0, 0, 1};
                    float t = top[0], sum = vsum[0], v[E];
#pragma unroll
                    for (int k = 0; k < RW; ++k)
                        if (k == i) {
                            t = top[k];
                            sum = vsum[k];
#pragma unroll
                            for (int e = 0; e < E; ++e) v[e] = qv[k][e];
                        }
                    tree_onto<E>(before, t, sum, v);
#pragma unroll
                    for (int k = 0; k < RW; ++k)
                        if (k == i) {
                            top[k] = t;
                            vsum[k] = sum;
#pragma unroll
                            for (int e = 0; e < E; ++e) qv[k][e] = v[e];
                        }
                } else {
                    const float2 x = *from_ml;
                    if (r >= rows || x.x == -INFINITY) continue;
#pragma unroll
                    for (int k = 0; k < RW; ++k)
                        if (k == i) {
                            const float t = fmaxf(top[k], x.x), f = ex2(x.x - t), g0 = top[k] == -INFINITY ? 0.f : ex2(top[k] - t);
#pragma unroll
                            for (int e = 0; e < E; ++e) qv[k][e] = (g0 == 0.f ? 0.f : qv[k][e] * g0) + from[e] * f;
                            vsum[k] = (g0 == 0.f ? 0.f : vsum[k] * g0) + x.y * f;
                            top[k] = t;
                        }
                }
            }
        }
        const bool finish = w.whole && !out_pass(p);
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const float il = finish ? (vsum[i] == 0.f ? 0.f : 1.f / vsum[i]) : 1.f;
#pragma unroll
            for (int e = 0; e < E; ++e) qv[i][e] *= il;
        }
        if (finish && !(p.flags & RQ_ATTN_ROTATED_OUT)) {
#pragma unroll
            for (int i = 0; i < RW; ++i) warp_rotate<E>(qv[i], sg, lane, !signs_first, inv_sqrt_dim<D>());
        }
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            const int r = i * kCWarps + warp, gr = w.mt * ROWS + r;
            if (r >= rows) break;
            if (finish) {
                const int64_t o = ((w.s.row0 + gr / p.group) * p.kv_heads + w.h) * p.group + gr % p.group;
#pragma unroll
                for (int e = 0; e < E; ++e) store_elem<IN>(p.out, o * D + lane * E + e, qv[i][e]);
            } else {
                float *to = part + (slot * ROWS + r) * D;
                float2 *to_ml = reinterpret_cast<float2 *>(ml + (slot * ROWS + r) * 2);
                if constexpr (P::kPass) {
                    if (w.whole) {
                        const int64_t o = tree_state<ROWS>(p, w.s.row0, w.mt, w.h, r);
                        to = p.state + o * D;
                        to_ml = p.state_ml + o;
                    }
                }
#pragma unroll
                for (int e = 0; e < E; ++e) to[lane * E + e] = qv[i][e];
                if (lane == 0) *to_ml = make_float2(top[i], vsum[i]);
            }
        }
        cta_sync();                                          // s.acc and s.q are free again
    }
    if constexpr (P::kPass) pass_wait();
}

template <int IN, int D, int ROWS, class P>
cudaError_t launch_tree_d(P &p, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t stream) {
    auto kern = attn_tree_mma_kernel<IN, D, ROWS, P>;
    const size_t smem = sizeof(MSmem<IN, D, ROWS>) + 1024;
    static std::atomic<uint64_t> allowed;
    cudaError_t e = allow_smem((const void *)kern, smem, allowed);
    if (e != cudaSuccess) return e;
    if constexpr (P::kPass) p.out_rows = p.out_pass ? ROWS : p.out_rows;
    e = launch_tree_kernel(kern, p, kMThreads, smem, stream, mk, mv, p);
    if (e != cudaSuccess) return e;
    if constexpr (P::kPass) {
        if (p.out_pass && p.place) return cudaSuccess;      // the pass after it joins
    }
    return launch_tree_join<IN, D, ROWS>(p, stream);
}

template <int IN, int ROWS, class P>
cudaError_t launch_tree_in(P &p, int64_t d, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t stream) {
    switch (d) {
        case 32: return launch_tree_d<IN, 32, ROWS>(p, mk, mv, stream);
        case 64: return launch_tree_d<IN, 64, ROWS>(p, mk, mv, stream);
        case 128: return launch_tree_d<IN, 128, ROWS>(p, mk, mv, stream);
        default: return launch_tree_d<IN, 256, ROWS>(p, mk, mv, stream);
    }
}

// The call's blocks of 8 or 16 rows; p as tree_params left it.
template <class P>
cudaError_t launch_tree_mma(const TreeCall &c, P &p, cudaStream_t stream) {
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorUnknown;
    const int rows = tree_rows(c) <= 8 ? 8 : 16;
    const int per_sm = blocks_per_sm(rows, c.head_dim);
    tree_ctas(c, p, rows, kTT, per_sm * sms);
    CUtensorMap mk, mv;
    if (!tree_maps(c, kTT, mk, mv)) return cudaErrorInvalidValue;
    const bool side = rows == 8;
    switch (c.in_type) {
        case IN_F32: return side ? launch_tree_in<IN_F32, 8>(p, c.head_dim, mk, mv, stream) : launch_tree_in<IN_F32, 16>(p, c.head_dim, mk, mv, stream);
        case IN_BF16: return side ? launch_tree_in<IN_BF16, 8>(p, c.head_dim, mk, mv, stream) : launch_tree_in<IN_BF16, 16>(p, c.head_dim, mk, mv, stream);
        default: return side ? launch_tree_in<IN_F16, 8>(p, c.head_dim, mk, mv, stream) : launch_tree_in<IN_F16, 16>(p, c.head_dim, mk, mv, stream);
    }
}

}  // namespace
}  // namespace rq
