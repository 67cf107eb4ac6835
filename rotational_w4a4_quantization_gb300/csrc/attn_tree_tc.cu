// attn_tree_tc.cu -- tree attention over the paged rotated INT4 cache on the
// 5th-generation tensor cores (sm_103a): blocks of 128 or 256 query rows.
//
// The same operator as attn_tree.cu (see there for the formulas).  Here the rows
// (nodes x query heads of a KV head) fill the 128 lanes of a tcgen05 MMA:
//   S = Q K^T   M128 N128 (tokens) K = D,  A = q~ in shared memory, fp16
//   O += P V    M128 N = D  K128 (tokens), A = P in tensor memory, fp16
// and a tile is 128 tokens.  Two score buffers: while the tensor core runs P V and the
// next Q K^T for one, 256 softmax threads, two to a row, turn the other's scores into
// weights.
//   NT = 2: 256 rows, buffer t has rows 128 t ..; every tile is used by both.
//   NT = 1: 128 rows; the tiles take the buffers in turn, each buffer with an accumulator
//           of its own, and the two are joined at the end.
//
// Roles (20 warps of which two idle, one block per SM):
//   warp 0       scales of each tile: their units, and the scales themselves where they
//                are not folded in
//   warp 1       tensor memory, all MMAs (one lane)
//   warps 4-11   softmax: warps 4-7 the first half of a tile's tokens, 8-11 the second;
//                the two threads of a row agree on its reference
//   warps 12-19  converters, two teams in turn: packed codes, loaded two operands ahead
//                straight into registers, -> fp16 in the 128-byte-swizzled operand
//                layout.  One layout serves both products: rows of 64 dims per token
//                are K-major for Q K^T and MN-major for P V.
// Tensor memory, 512 columns: S0 S1 (128 each; the weights of each half overwrite the first
// half of its scores) and O0 O1 (D each).
//
// Scales.  With bf16 queries they are folded into the operands: k^ and v^ as fp16(code *
// scale), scales relative to a power of two per tile, one rounding (the scale enters in
// two fp16 parts).  The softmax then reads nothing but its scores: broadcasting scales from
// shared memory costs 4 cycles per 16 bytes and warp, and bound the kernel (8 warps x 64
// loads per tile; measured 2,150 cycles per tile for that softmax alone, against 2,048 of
// MMAs).
// A tile keeps exact codes if a scale of it is not finite or they lie too far apart (values
// by more than 2^8, keys 2^12), and applies them to scores and weights, so that a large
// scale costs the others no bits and what an unseen token holds (a NaN scale, say) reaches
// nobody.  Where every tile does so, 64 nodes of 16 sequences of 16k take 766 us (bf16) for
// 330, 16 nodes of 4k 155 (fp16) for 104.  fp16 queries, whose outputs resolve an 11-bit rounding of q~, k^ and v^, keep q~
// in two fp16 parts (Q K^T runs twice) and the scales out of the operands; the weights with
// vs in them round once (16 sequences of up to 4k: outputs 3.0e-4 off; with the scales of V
// folded 3.3e-4, and 2 us slower).
//
// Weights: P = 2^(s - M + ev) (2^ev the tile's unit of vs) is what the MMA sees, rounded
// to fp16; the sum l adds 2^(s - M) in fp32.  O / l does not depend on M, so M only has
// to keep P in range: it moves only when some P would pass 2^15, and then puts it at 2^9
// (the accumulator is then rescaled in place, between the commit that delivers S and the
// arrival that delivers P, when no MMA touches it).  fp16 keeps 11 bits down to 2^-14, so
// of tokens at least 23 bits below the largest, and something down to 2^-25.
//
// Measured (D = 128): 256 rows (bf16, 16 sequences of up to 32k, 8 KV heads): 426 us, 0.69
// PFLOP/s of Q K^T and P V, where the products alone take 153; a tile takes 5,000 cycles
// of which the MMAs run 2,048.  The softmax bounds it: 1,800 cycles for half a tile, most
// of it latency of tensor-memory loads, exponentials and the exchange between a row's
// threads (issue slots are two fifths full), and 800 from one half to the next.  Slower
// were, with one limit of 96 registers for all warps: one pass over the scores with the old
// reference, weights kept back in registers (431 us); scores kept in registers (457,
// spills); 32 columns a load (433); buffers of 64 columns (423, as Q K^T with N = 64 takes
// 48 cycles for 32's work).  64 rows (fp16, 16 sequences of up to 4k): 72 us, where the
// bytes take 9: starts and ends of units; with a buffer per softmax team, 128 columns to a
// thread, 86 (and the 256 rows 404).
#include "rq.h"
#include "rq_internal.h"
#include "tree_device.cuh"

namespace rq {
namespace {

constexpr int kTcTT = 128;               // tokens per tile
constexpr int kHT = kTcTT / 2;           // of which a softmax thread has half
constexpr int kOps = 4;                  // operand slots
constexpr int kSc = 4;                   // scale slots
constexpr int kSoftWarps = 8, kConvTeams = 2, kTeamWarps = 4, kConvWarps = kConvTeams * kTeamWarps;
constexpr int kTcThreads = 32 * (4 + kSoftWarps + kConvWarps);

template <int D, int NT, int HV>
struct TSmem {
    static constexpr int PANEL = 128 * 128;                 // 128 rows x 64 dims of fp16
    static constexpr int TILE = D / 64 * PANEL;
    alignas(1024) uint8_t q[NT * HV][TILE];
    alignas(1024) uint8_t op[kOps][TILE];
    alignas(16) float ks[kSc][kTcTT];
    alignas(16) float vs[kSc][kTcTT];
    float2 unit[kSc];                                       // a tile's 2^ek and ev; 0 and 0: scales not folded in
    float rfac[NT * 128];                                   // s = rfac S (times ks)
    float best[2][2][128], sum[2][2][128];                  // what the two threads of a row tell each other: [buffer][team], [team][buffer]
    TreeLine line;
    TreeWork work[2];                                       // each softmax team's copy of the stretch: kept here, not in registers
    alignas(8) uint64_t sc_full[kSc], sc_empty[kSc];
    uint64_t op_full[kOps], op_empty[kOps];
    uint64_t q_full, s_full[2], p_full[2], p_free[2], o_full[2];
    uint32_t valid[kSc];                                    // bit c: tokens 16 c .. lie on a page of the cache
    uint32_t sign_words[8];
    uint32_t tmem_base;
    volatile int abort_flag;
};

// Shared-memory matrix descriptor, 128-byte swizzle.  K-major (Q, K): groups of 8 rows
// 1024 bytes apart.  MN-major (V): 8-token groups 1024 bytes apart, panels of 64 dims
// PANEL bytes apart.
__device__ __forceinline__ uint64_t op_desc(uint32_t saddr, uint32_t lead_bytes) {
    return (uint64_t)((saddr >> 4) & 0x3FFF) | ((uint64_t)(lead_bytes >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
// kind::f16, fp16 operands, fp32 accumulator, M = 128
__device__ __forceinline__ constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
    return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
                 "r"((uint32_t)acc)
                 : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
                 "r"((uint32_t)acc)
                 : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(t_smem(bar)) : "memory");
}
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

#define RQ_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), "=r"(a[i + 6]), "=r"(a[i + 7])
#define RQ_W8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), "r"(a[i + 6]), "r"(a[i + 7])
__device__ __forceinline__ void tm_ld8(uint32_t t, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : RQ_R8(r, 0) : "r"(t));
}
__device__ __forceinline__ void tm_ld16(uint32_t t, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : RQ_R8(r, 0), RQ_R8(r, 8) : "r"(t));
}
__device__ __forceinline__ void tm_ld32(uint32_t t, uint32_t *r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
                 "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
                 : RQ_R8(r, 0), RQ_R8(r, 8), RQ_R8(r, 16), RQ_R8(r, 24) : "r"(t));
}
__device__ __forceinline__ void tm_st8(uint32_t t, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), RQ_W8(r, 0) : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t t, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
                 "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(t),
                 RQ_W8(r, 0), RQ_W8(r, 8), RQ_W8(r, 16), RQ_W8(r, 24) : "memory");
}
// Waits for the loads before it; the registers pass through it, so that no use of them
// is scheduled ahead of the wait.
#define RQ_P8(a, i) "+r"(a[i]), "+r"(a[i + 1]), "+r"(a[i + 2]), "+r"(a[i + 3]), "+r"(a[i + 4]), "+r"(a[i + 5]), "+r"(a[i + 6]), "+r"(a[i + 7])
__device__ __forceinline__ void tc_wait_ld8(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : RQ_P8(r, 0) : : "memory");
}
__device__ __forceinline__ void tc_wait_ld16(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : RQ_P8(r, 0), RQ_P8(r, 8) : : "memory");
}
__device__ __forceinline__ void tc_wait_ld32(uint32_t *r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : RQ_P8(r, 0), RQ_P8(r, 8), RQ_P8(r, 16), RQ_P8(r, 24) : : "memory");
}
#undef RQ_R8
#undef RQ_W8
#undef RQ_P8

// The order in which code tiles are loaded, converted and used, for a stretch of T
// tiles.  NT = 2: K0 V0 K1 V1 ...; NT = 1: K0 K1 V0 K2 V1 ... K(T-1) V(T-2) V(T-1).
template <int NT>
__device__ __forceinline__ void item_at(int i, int T, int &tile, bool &is_v) {
    if (NT == 2) {
        tile = i >> 1;
        is_v = i & 1;
    } else if (i == 0) {
        tile = 0;
        is_v = false;
    } else if (i == 2 * T - 1) {
        tile = T - 1;
        is_v = true;
    } else {
        is_v = !(i & 1);
        tile = is_v ? (i >> 1) - 1 : (i + 1) >> 1;
    }
}
template <int NT>
__device__ __forceinline__ int item_of_k(int k) { return NT == 2 ? 2 * k : (k == 0 ? 0 : 2 * k - 1); }
template <int NT>
__device__ __forceinline__ int item_of_v(int k, int T) { return NT == 2 ? 2 * k + 1 : (k == T - 1 ? 2 * T - 1 : 2 * k + 2); }

// A word of 8 codes as 8 fp16 operands code * (hi + lo), rounded once, in the order of
// the dims 0 4 1 5 2 6 3 7.  0x6400 | u is 1024 + u, so nibbles 0 and 4 (u = code + 8
// after the sign bit's flip) lose 1032; nibbles 1 and 5, which stay four bits up, are
// 1024 + 16 u: times 1/16, less 72.  Both exact.
__device__ __forceinline__ uint4 operands(uint32_t x, __half2 hi, __half2 lo) {
    const __half2 m0 = __half2half2(__ushort_as_half(0xe408)), r16 = __half2half2(__ushort_as_half(0x2c00)),
                  m1 = __half2half2(__ushort_as_half(0xd480));             // -1032, 1/16, -72
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        const uint32_t y = x >> (4 * j);
        const uint32_t a = (y & 0x000f000fu) ^ 0x64086408u, b = (y & 0x00f000f0u) ^ 0x64806480u;
        const __half2 ca = __hadd2(*reinterpret_cast<const __half2 *>(&a), m0);
        const __half2 cb = __hfma2(*reinterpret_cast<const __half2 *>(&b), r16, m1);
        const __half2 ha = __hfma2(ca, hi, __hmul2(ca, lo)), hb = __hfma2(cb, hi, __hmul2(cb, lo));
        r[j] = *reinterpret_cast<const uint32_t *>(&ha);
        r[j + 1] = *reinterpret_cast<const uint32_t *>(&hb);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
// The exponent e >= least with 2^e above the largest of a tile's 128 scales (`none` where all
// are 0): one warp, four scales a lane.  Scales are not negative, so their bits order them.
__device__ __forceinline__ int tile_exponent(const float4 &x, int least, int none) {
    const uint32_t top = __reduce_max_sync(0xffffffffu, max(max(__float_as_uint(x.x), __float_as_uint(x.y)),
                                                            max(__float_as_uint(x.z), __float_as_uint(x.w))));
    return top == 0 ? none : max(least, min((int)((top >> 23) & 255u) - 126, 100));
}
// The first n of four scales are within 2^(bits + 1) of 2^e, and finite, or 0 where that may be.
__device__ __forceinline__ bool of_a_kind(const float4 &x, int n, int e, int bits, bool zeros) {
    const float lo = __uint_as_float((uint32_t)(127 + max(e - 1 - bits, -120)) << 23), hi = __uint_as_float((uint32_t)(127 + e) << 23);
    auto ok = [&](float v, int i) { return i >= n || (v >= lo && v <= hi) || (zeros && v == 0.f); };
    return ok(x.x, 0) && ok(x.y, 1) && ok(x.z, 2) && ok(x.w, 3);
}
// How far apart a tile's scales may lie to share a unit: the products of keys keep 11 bits in
// fp16; values may cost the weights' range that much, as a row's reference takes a tile's
// largest score and largest value scale for one token's.  So a value row of zeros is not of
// a kind with others either: it may be the one with the score.
constexpr int kKeyBits = 12, kValueBits = 8;
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }   // |e| <= 126
__device__ __forceinline__ uint4 ld_once(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ float max3(float a, float b, float c) { return fmaxf(fmaxf(a, b), c); }

__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
// t_mbar_wait by a whole warp, with one answer
__device__ __forceinline__ bool warp_wait(uint64_t *b, uint32_t parity, volatile int *abort_flag, int *err) {
    return __all_sync(0xffffffffu, t_mbar_wait(b, parity, abort_flag, err));
}

// position p of an 8-group of operand columns holds dim kPerm(p) of the group
__device__ __forceinline__ constexpr int perm8(int p) { return (p & 1) * 4 + (p >> 1); }

// Cache row of token t of a work's KV head, -1 past the sequence or off the cache.
__device__ __forceinline__ int64_t tree_row(const TreeParams &p, const TreeWork &w, int t) {
    if (t >= w.s.len) return -1;
    const int64_t pg = p.table[w.b * p.width + (t >> p.log_page)];
    if (pg < 0 || pg >= p.pages) return -1;
    return ((pg * p.kv_heads + w.h) << p.log_page) + (t & ((1 << p.log_page) - 1));
}

constexpr int kCW = 16;                  // scores that a row works on at a time: more of them spill

// One row's state: the reference M (-inf: nothing seen yet) and the sum l.
struct SoftRow {
    float M, l;
};

// One row's 128 scores of a tile -> weights over them in tensor memory.  Two passes over
// the scores, the next kCW always on their way: the largest first, so that M is settled
// once for the tile and the second pass has neither votes nor branches (settling it per
// chunk cost 200 cycles each); returns the factor that earlier tiles' sums need.
//   s = a S;  weight = 2^(s - M + ev).  KS: the operands are exact codes, s = a S ks and
//   the weights carry vs (relative to 2^ev).
// MASK: vis has a bit per token; the loops stay rolled, as few tiles come here.
template <bool KS, bool MASK, class X>
__device__ __forceinline__ float soft_tile(uint32_t tS, const float *ks, const float *vs, float a, float ev, uint32_t vis0, uint32_t vis1,
                                           SoftRow &r, const X &both) {
    constexpr int C = kHT / kCW, UNROLL = MASK ? 1 : C / 2;
    auto seen = [&](int c) { return (c & 2 ? vis1 : vis0) >> (kCW * (c & 1)); };
    uint32_t s0[kCW], s1[kCW];
    tm_ld16(tS, s0);
    float top0 = -INFINITY, top1 = -INFINITY;
    auto largest = [&](const uint32_t (&x)[kCW], int c) {
#pragma unroll
        for (int i = 0; i < kCW; i += 4) {
            float4 v = make_float4(__uint_as_float(x[i]), __uint_as_float(x[i + 1]), __uint_as_float(x[i + 2]), __uint_as_float(x[i + 3]));
            if constexpr (KS) {
                const float4 k = *reinterpret_cast<const float4 *>(ks + kCW * c + i);
                v.x *= k.x;
                v.y *= k.y;
                v.z *= k.z;
                v.w *= k.w;
            }
            if constexpr (MASK) {
                const uint32_t w = seen(c) >> i;
                v = make_float4(w & 1 ? v.x : -INFINITY, w & 2 ? v.y : -INFINITY, w & 4 ? v.z : -INFINITY, w & 8 ? v.w : -INFINITY);
            }
            top0 = max3(top0, v.x, v.y);
            top1 = max3(top1, v.z, v.w);
        }
    };
#pragma unroll(UNROLL)
    for (int c = 0; c < C; c += 2) {
        tc_wait_ld16(s0);
        tm_ld16(tS + kCW * (c + 1), s1);
        largest(s0, c);
        tc_wait_ld16(s1);
        tm_ld16(tS + kCW * ((c + 2) % C), s0);                    // at the end: the first again
        largest(s1, c + 1);
    }
    const float best = both(fmaxf(top0, top1) * a + ev);          // a >= 0
    float f = 1.f;
    if (best > r.M + kWeightMost) {                               // also the first time, where M = -inf
        if (r.M != -INFINITY) f = ex2(r.M - (best - kWeightTo));
        r.M = best - kWeightTo;
        r.l *= f;
    }
    const float Mz = (r.M == -INFINITY ? 0.f : r.M) - ev;
    const float2 a2 = make_float2(a, a), nm = make_float2(-Mz, -Mz);
    float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
    auto weigh = [&](const uint32_t (&x)[kCW], int c) {
        uint32_t pk[kCW / 2];
#pragma unroll
        for (int i = 0; i < kCW / 2; i += 2) {
            float2 t0 = make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
            float2 t1 = make_float2(__uint_as_float(x[2 * i + 2]), __uint_as_float(x[2 * i + 3]));
            if constexpr (KS) {
                const float4 k = *reinterpret_cast<const float4 *>(ks + kCW * c + 2 * i);
                t0 = __ffma2_rn(__fmul2_rn(t0, a2), make_float2(k.x, k.y), nm);
                t1 = __ffma2_rn(__fmul2_rn(t1, a2), make_float2(k.z, k.w), nm);
            } else {
                t0 = __ffma2_rn(t0, a2, nm);
                t1 = __ffma2_rn(t1, a2, nm);
            }
            if constexpr (MASK) {
                const uint32_t w = seen(c) >> (2 * i);
                t0 = make_float2(w & 1 ? t0.x : -INFINITY, w & 2 ? t0.y : -INFINITY);
                t1 = make_float2(w & 4 ? t1.x : -INFINITY, w & 8 ? t1.y : -INFINITY);
            }
            const float2 p0 = make_float2(ex2(t0.x), ex2(t0.y)), p1 = make_float2(ex2(t1.x), ex2(t1.y));
            sum0 = __fadd2_rn(sum0, p0);
            sum1 = __fadd2_rn(sum1, p1);
            float2 w0 = p0, w1 = p1;
            if constexpr (KS) {
                const float4 v = *reinterpret_cast<const float4 *>(vs + kCW * c + 2 * i);
                w0 = __fmul2_rn(p0, make_float2(v.x, v.y));
                w1 = __fmul2_rn(p1, make_float2(v.z, v.w));
            }
            const __half2 h0 = __floats2half2_rn(w0.x, w0.y), h1 = __floats2half2_rn(w1.x, w1.y);
            pk[i] = *reinterpret_cast<const uint32_t *>(&h0);
            pk[i + 1] = *reinterpret_cast<const uint32_t *>(&h1);
        }
        tm_st8(tS + kCW / 2 * c, pk);
    };
    // the columns of a chunk are overwritten by the weights of twice its number at the earliest
#pragma unroll(UNROLL)
    for (int c = 0; c < C; c += 2) {
        tc_wait_ld16(s0);
        tm_ld16(tS + kCW * (c + 1), s1);
        weigh(s0, c);
        tc_wait_ld16(s1);
        if (c + 2 < C) tm_ld16(tS + kCW * (c + 2), s0);
        weigh(s1, c + 1);
    }
    const float2 s2 = __fadd2_rn(sum0, sum1);
    r.l += (s2.x + s2.y) * ex2(-ev);
    return f;
}

// The tokens of half a tile that a row's node sees, a bit each: a warp reads a node's 32
// mask bytes together, and the rows of that node keep the ballot.
//   node: this row's, node0, node1: the warp's first and last; valid: bit c says that
//   tokens 16 c .. lie on a page of the cache.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }
__device__ __forceinline__ void tree_visible(const TreeParams &p, const TreeSeq &q, int node, int node0, int node1, int t0,
                                             uint32_t valid, uint32_t &vis0, uint32_t &vis1) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int g = 0; g < kHT / 32; ++g) {
        const int t = t0 + 32 * g, j = t + lane - q.ctx;
        uint32_t seen = 0;
        if (!p.mask) {
            seen = below(node + 1 + q.ctx - t);
        } else if (t + 32 <= q.ctx) {
            seen = 0xffffffffu;
        } else if (t < q.len) {
            const uint8_t *m = p.mask + q.row0 * p.mask_stride + j;
            const bool in = j >= 0 && j < q.n;
#pragma unroll 8
            for (int nd = node0; nd <= node1; ++nd) {
                const uint32_t b = __ballot_sync(0xffffffffu, j < 0 || (in && m[nd * p.mask_stride] != 0));
                if (nd == node) seen = b;
            }
        }
        const uint32_t v = valid >> (2 * g);
        seen &= below(q.len - t) & ((v & 1 ? 0xffffu : 0u) | (v & 2 ? 0xffff0000u : 0u));
        vis0 = vis1;
        vis1 = node < q.n ? seen : 0u;
    }
}

// A tile with exact codes, where some scale is not finite or the scales lie too far apart
// to share a unit: s = a S ks, weight = 2^(s - M) vs.  M follows the largest
// s + log2 vs, the weight's exponent.  A masked weight is zero whatever its scales hold.
// Hardly a tile comes here, and its time is the fetching of code that ran for none
// before: the loops stay rolled.
template <class X>
__device__ __forceinline__ float soft_exact(uint32_t tS, const float *ks, const float *vs, float a, uint32_t vis0, uint32_t vis1,
                                            SoftRow &r, const X &both) {
    uint32_t x[kCW];
    float best = -INFINITY, only = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < kHT / kCW; ++c) {
        const uint32_t w = (c & 2 ? vis1 : vis0) >> (kCW * (c & 1));
        tm_ld16(tS + kCW * c, x);
        tc_wait_ld16(x);
#pragma unroll
        for (int i = 0; i < kCW; ++i) {
            const bool sees = (w >> i) & 1;
            const float sc = sees ? __uint_as_float(x[i]) * a * ks[kCW * c + i] : -INFINITY;
            only = fmaxf(only, sc);
            best = fmaxf(best, sees ? sc + lg2(vs[kCW * c + i]) : -INFINITY);
        }
    }
    best = both(fmaxf(best, only + kLeastValue));                       // rows of zero values: keeps 2^(s - M) itself finite
    float f = 1.f;
    if (best > r.M + kWeightMost) {
        if (r.M != -INFINITY) f = ex2(r.M - (best - kWeightTo));
        r.M = best - kWeightTo;
        r.l *= f;
    }
    const float Mz = r.M == -INFINITY ? 0.f : r.M;
#pragma unroll 1
    for (int c = 0; c < kHT / kCW; ++c) {
        const uint32_t w = (c & 2 ? vis1 : vis0) >> (kCW * (c & 1));
        tm_ld16(tS + kCW * c, x);
        tc_wait_ld16(x);
        uint32_t pk[kCW / 2];
#pragma unroll
        for (int i = 0; i < kCW; i += 2) {
            float pw[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const bool sees = (w >> (i + j)) & 1;
                const float e = sees ? ex2(__uint_as_float(x[i + j]) * a * ks[kCW * c + i + j] - Mz) : 0.f;
                r.l += e;
                pw[j] = sees ? e * vs[kCW * c + i + j] : 0.f;
            }
            const __half2 h = __floats2half2_rn(pw[0], pw[1]);
            pk[i / 2] = *reinterpret_cast<const uint32_t *>(&h);
        }
        tm_st8(tS + kCW / 2 * c, pk);
    }
    return f;
}

template <int IN, int D, int NT, int HV>
__global__ void __launch_bounds__(kTcThreads, 1)
attn_tree_tc_kernel(const __grid_constant__ TreeParams p) {
    using S = TSmem<D, NT, HV>;
    constexpr int ROWS = 128 * NT, RB = D / 2;
    constexpr bool FOLD = HV == 1;                     // the scales go into the operands
    extern __shared__ uint8_t raw[];
    S &s = *reinterpret_cast<S *>(raw + ((1024u - (t_smem(raw) & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kSc; ++i) {
            t_mbar_init(&s.sc_full[i], 1);
            t_mbar_init(&s.sc_empty[i], kSoftWarps + kTeamWarps);
        }
        for (int i = 0; i < kOps; ++i) {
            t_mbar_init(&s.op_full[i], kTeamWarps);
            t_mbar_init(&s.op_empty[i], 1);
        }
        t_mbar_init(&s.q_full, kSoftWarps);
        for (int i = 0; i < 2; ++i) {
            t_mbar_init(&s.s_full[i], 1);
            t_mbar_init(&s.p_full[i], kSoftWarps);
            t_mbar_init(&s.p_free[i], 1);
            t_mbar_init(&s.o_full[i], 1);
        }
        s.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(t_smem(&s.tmem_base)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    block_sign_words<D>(s.sign_words, p.seed);
    tree_join_may_begin();
    tc_fence_before();
    tree_scan<ROWS, kTcTT>(p, s.line);               // ends with a block barrier
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    const uint32_t tO[2] = {tmem + 256, tmem + 256 + (uint32_t)D};
    const int64_t total = s.line.prefix[kScan];
    const int64_t begin = tree_begin(total, p.ctas, blockIdx.x), end = tree_begin(total, p.ctas, blockIdx.x + 1);

    if (warp == 0) {
        // ---------------- scales ----------------
        uint32_t sc = 0;
        TreeJoin join{};
        for (int64_t at = begin; at < end;) {
            const TreeWork w = tree_work<ROWS, kTcTT>(p, s.line, at, begin, end);
            const int T = w.t1 - w.t0;
            at += w.used;
            if (T <= 0) continue;
            // lane l: tokens 4 l .. 4 l + 3 of a tile, the next tile's loaded ahead
            float4 nk, nv;
            int nthere;
            auto load = [&](int k) {
                const int64_t row = k < T ? tree_row(p, w, (w.t0 + k) * kTcTT + 4 * lane) : -1;
                nthere = 0;
                nk = nv = make_float4(0.f, 0.f, 0.f, 0.f);
                if (row >= 0) {
                    nk = *reinterpret_cast<const float4 *>(p.ks + row);
                    nv = *reinterpret_cast<const float4 *>(p.vs + row);
                    const int left = w.s.len - ((w.t0 + k) * kTcTT + 4 * lane);   // past the sequence: none
                    nthere = min(left, 4);
                    if (left < 4) {
                        nk = make_float4(nk.x, left > 1 ? nk.y : 0.f, left > 2 ? nk.z : 0.f, 0.f);
                        nv = make_float4(nv.x, left > 1 ? nv.y : 0.f, left > 2 ? nv.z : 0.f, 0.f);
                    }
                }
            };
            load(0);
            for (int k = 0; k < T; ++k, ++sc) {
                const uint32_t scs = sc % kSc;
                const float4 ck = nk, cv = nv;
                const int there = nthere;
                load(k + 1);
                const uint32_t quads = __ballot_sync(0xffffffffu, there > 0);
                // a tile of zero values moves no row's reference: its unit is the least
                const int ek = FOLD ? tile_exponent(ck, -100, 0) : 0, ev = tile_exponent(cv, (int)kLeastValue, (int)kLeastValue);
                // scales that are not of a kind stay out of the operands and the tile's unit
                const bool nothing = __all_sync(0xffffffffu, cv.x == 0.f && cv.y == 0.f && cv.z == 0.f && cv.w == 0.f);
                const bool exact = __any_sync(0xffffffffu, !((!FOLD || of_a_kind(ck, there, ek, kKeyBits, true)) &&
                                                             of_a_kind(cv, there, ev, kValueBits, nothing)));
                uint32_t chunks = 0;
#pragma unroll
                for (int c = 0; c < 8; ++c) chunks |= ((quads >> (4 * c)) & 1) << c;
                warp_wait(&s.sc_empty[scs], ((sc / kSc) & 1) ^ 1, &s.abort_flag, p.err);
                if (!FOLD || exact) {
                    const float down = exact ? 1.f : pow2(-ev);
                    reinterpret_cast<float4 *>(s.ks[scs])[lane] = ck;
                    reinterpret_cast<float4 *>(s.vs[scs])[lane] = make_float4(cv.x * down, cv.y * down, cv.z * down, cv.w * down);
                }
                if (lane == 0) {
                    s.unit[scs] = exact ? make_float2(0.f, 0.f) : make_float2(pow2(ek), (float)ev);
                    s.valid[scs] = chunks;
                }
                __syncwarp();
                if (lane == 0) t_mbar_arrive(&s.sc_full[scs]);
            }
            tree_note<ROWS, D>(p, s.line, w, begin, end, join);
        }
        tree_noted<ROWS, D>(p, join);
    } else if (warp == 1) {
        // ---------------- MMA ----------------
        // The whole warp runs the loop, so that descriptors stay in uniform registers;
        // one lane issues (16 MMAs of 64 cycles each per tile leave no time for more).
        const bool one = elect_one();
        uint32_t base = 0, unit = 0, pc[2] = {0, 0}, fc[2] = {0, 0};   // items of earlier stretches; stretches; weights per buffer, those given up
        constexpr uint32_t id_qk = idesc_f16(kTcTT, false), id_pv = idesc_f16(D, true);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dq = op_desc(t_smem(s.q[0]), 16), dk = op_desc(t_smem(s.op[0]), 16);
        const uint64_t dv = op_desc(t_smem(s.op[0]), S::PANEL);
        bool ok = true;
        for (int64_t at = begin; at < end && ok; ++unit) {
            const TreeWork w = tree_work<ROWS, kTcTT>(p, s.line, at, begin, end);
            const int T = __shfl_sync(0xffffffffu, w.t1 - w.t0, 0), J = NT * T;
            at += w.used;
            if (T <= 0) continue;
            ok = warp_wait(&s.q_full, unit & 1, &s.abort_flag, p.err);
            auto qk = [&](int j) {
                const int k = NT == 2 ? j >> 1 : j, t = j & 1;
                const uint32_t i = base + item_of_k<NT>(k), slot = i % kOps;
                if (NT == 1 || t == 0) ok = ok && warp_wait(&s.op_full[slot], (i / kOps) & 1, &s.abort_flag, p.err);
                if (!ok) return;
                tc_fence_after();
                const uint64_t b = dk + slot * (S::TILE >> 4);
                const uint64_t a = dq + (NT == 2 ? t * (S::TILE >> 4) : 0);
                if (one) {
#pragma unroll
                    for (int hv = 0; hv < HV; ++hv)
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) {
                            const uint32_t off = ((c >> 2) * S::PANEL + (c & 3) * 32) >> 4;
                            mma_ss(tm + 128 * t, a + hv * (S::TILE >> 4) + off, b + off, id_qk, hv + c > 0);
                        }
                    if (NT == 1 || t == 1) tc_commit(&s.op_empty[slot]);
                    tc_commit(&s.s_full[t]);
                }
                __syncwarp();
            };
            qk(0);
            if (J > 1) qk(1);
            for (int j = 0; j < J && ok; ++j) {
                const int k = NT == 2 ? j >> 1 : j, t = j & 1;
                const uint32_t i = base + item_of_v<NT>(k, T), slot = i % kOps;
                if (NT == 1 || t == 0) ok = ok && warp_wait(&s.op_full[slot], (i / kOps) & 1, &s.abort_flag, p.err);
                ok = ok && warp_wait(&s.p_full[t], pc[t] & 1, &s.abort_flag, p.err);
                ++pc[t];
                if (!ok) break;
                tc_fence_after();
                const uint64_t b = dv + slot * (S::TILE >> 4);
                if (one) {
#pragma unroll
                    for (int c = 0; c < kTcTT / 16; ++c)
                        mma_ts(tm + 256 + D * t, tm + 128 * t + (c < 4 ? 8 * c : 64 + 8 * (c - 4)), b + c * (2048 >> 4), id_pv, j >= 2 || c > 0);
                    if (NT == 1 || t == 1) tc_commit(&s.op_empty[slot]);
                    tc_commit(j + 2 < J ? &s.p_free[t] : &s.o_full[t]);
                }
                __syncwarp();
                // products of different shapes need not run in the order of their issue: the
                // weights are read before the next scores take their place
                if (j + 2 < J) {
                    ok = ok && warp_wait(&s.p_free[t], fc[t] & 1, &s.abort_flag, p.err);
                    ++fc[t];
                    qk(j + 2);
                }
            }
            base += 2 * T;
        }
    } else if (warp >= 4 && warp < 4 + kSoftWarps) {
        // ---------------- softmax: two teams, one per half of the tokens ----------------
        const int team = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;     // row of the 128
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        auto both_sync = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
        const bool signs_first = (p.flags & RQ_SIGNS_FIRST) != 0;
        auto team_sync = [&] { asm volatile("bar.sync %0, 128;" ::"r"(2 + team) : "memory"); };
        uint32_t sc = 0, uses = 0, units = 0;          // tiles so far; a bit per buffer: parity of its scores, of its finished sums
        const TreeWork &w = s.work[team];
        for (int64_t at = begin; at < end;) {
            if (quarter == 0) {
                const TreeWork x = tree_work<ROWS, kTcTT>(p, s.line, at, begin, end);
                if (lane == 0) s.work[team] = x;
            }
            team_sync();
            const int T = w.t1 - w.t0;
            at += w.used;
            if (T <= 0) continue;
            const int rows = min(ROWS, w.s.n * p.group - w.mt * ROWS);        // of the block

            // ---- q~: four threads to a row, a quarter of its dims each; butterflies in
            // registers but for two exchanges ----
            // 64 rows a pass; what lies in the tile beyond the last row's pass reaches no row that counts
#pragma unroll 1
            for (int pass = 0; pass * 64 < rows; ++pass) {
                constexpr int HD = D / 4;
                const int hf = threadIdx.x & 3, r = pass * 64 + ((threadIdx.x - 128) >> 2), rr = r & 127, gr = w.mt * ROWS + r;
                const char *src = static_cast<const char *>(p.q) + ((w.s.row0 + gr / p.group) * p.q_token +
                                  (w.h * p.group + gr % p.group) * p.q_head + hf * HD) * 2;
                float2 v[HD / 2];
#pragma unroll
                for (int i = 0; i < HD / 8; ++i) {
                    float f[8];
                    unpack16<IN>(r < rows ? reinterpret_cast<const uint4 *>(src)[i] : make_uint4(0u, 0u, 0u, 0u), f);
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[4 * i + e] = make_float2(f[2 * e], f[2 * e + 1]);
                }
                auto signs = [&] {
#pragma unroll
                    for (int i = 0; i < HD / 2; ++i) {
                        const uint32_t m = s.sign_words[(hf * HD + 2 * i) >> 5] >> ((hf * HD + 2 * i) & 31);
                        v[i].x = __uint_as_float(__float_as_uint(v[i].x) ^ (m << 31));
                        v[i].y = __uint_as_float(__float_as_uint(v[i].y) ^ ((m >> 1) << 31));
                    }
                };
                if (signs_first) signs();
#pragma unroll
                for (int i = 0; i < HD / 2; ++i) v[i] = make_float2(v[i].x + v[i].y, v[i].x - v[i].y);
#pragma unroll
                for (int st = 1; st < HD / 2; st <<= 1)
#pragma unroll
                    for (int i = 0; i < HD / 2; ++i)
                        if (!(i & st)) {
                            const float2 x = v[i], y = v[i + st];
                            v[i] = __fadd2_rn(x, y);
                            v[i + st] = __ffma2_rn(y, make_float2(-1.f, -1.f), x);
                        }
#pragma unroll
                for (int st = 1; st < 4; st <<= 1) {
                    const float sg = hf & st ? -1.f : 1.f;
#pragma unroll
                    for (int i = 0; i < HD / 2; ++i) {
                        const float2 o = make_float2(__shfl_xor_sync(0xffffffffu, v[i].x, st), __shfl_xor_sync(0xffffffffu, v[i].y, st));
                        v[i] = __ffma2_rn(v[i], make_float2(sg, sg), o);
                    }
                }
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < HD / 2; ++i) top = max3(top, fabsf(v[i].x), fabsf(v[i].y));
                if (!signs_first) signs();
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // top < 2^ex: q~ enters the MMA relative to that
                const int ex = max(-100, min((int)((__float_as_uint(top) >> 23) & 255u) - 126, 120));
                // the scale's sign goes into q~: the softmax takes the largest score for the largest product
                if (hf == 0) s.rfac[r] = pow2(ex) * inv_sqrt_dim<D>() * fabsf(p.score_scale);
                const float down = copysignf(pow2(-ex), p.score_scale);
                uint8_t *const dst = s.q[NT == 2 ? r >> 7 : 0] + rr * 128;
#pragma unroll
                for (int i = 0; i < HD / 8; ++i) {
                    uint32_t h[4], lo[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {          // dims j and j + 4 of the group
                        const float2 u0 = v[4 * i + (j >> 1)], u1 = v[4 * i + 2 + (j >> 1)];
                        const float x = (j & 1 ? u0.y : u0.x) * down, y = (j & 1 ? u1.y : u1.x) * down;
                        const __half2 hh = __floats2half2_rn(x, y);
                        h[j] = *reinterpret_cast<const uint32_t *>(&hh);
                        if constexpr (HV == 2) {
                            const float2 got = __half22float2(hh);
                            const __half2 ll = __floats2half2_rn(x - got.x, y - got.y);
                            lo[j] = *reinterpret_cast<const uint32_t *>(&ll);
                        }
                    }
                    const int d = hf * HD + 8 * i;
                    const uint32_t off = (d >> 6) * S::PANEL + ((((d & 63) >> 3) ^ (rr & 7)) << 4);
                    *reinterpret_cast<uint4 *>(dst + off) = make_uint4(h[0], h[1], h[2], h[3]);
                    if constexpr (HV == 2) *reinterpret_cast<uint4 *>(dst + S::TILE + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) t_mbar_arrive(&s.q_full);
            both_sync();
            // Both threads of a row take every score buffer, half of its columns each: while
            // the tensor core works for one buffer, all of them have the other.
            float fac = s.rfac[row], fac2 = s.rfac[NT == 2 ? 128 + row : row];
            SoftRow r{-INFINITY, 0.f}, r2{-INFINITY, 0.f};               // this buffer's, the other's
            const int J = NT * T;
            for (int j = 0; j < J; ++j) {
                const int k = NT == 2 ? j >> 1 : j, t = j & 1, blk = NT == 2 ? 128 * t : 0;
                const uint32_t scs = (sc + k) % kSc, tS = tmem + 128 * t + kHT * team + lanes;
                bool ok = t_mbar_wait(&s.sc_full[scs], ((sc + k) / kSc) & 1, &s.abort_flag, p.err);
                const int t0 = (w.t0 + k) * kTcTT + kHT * team;
                const float2 unit = s.unit[scs];
                const uint32_t valid = (s.valid[scs] >> (kHT / 16 * team)) & 15u;
                const float a = unit.x == 0.f ? fac : fac * unit.x, ev = unit.y;
                const bool plain = unit.x != 0.f && t0 + kHT <= w.s.ctx && valid == 15u;
                ok = t_mbar_wait(&s.s_full[t], (uses >> t) & 1, &s.abort_flag, p.err) && ok;
                ok = __all_sync(0xffffffffu, ok);
                uses ^= 1u << t;
                tc_fence_after();
                if (blk + quarter * 32 < rows) {                               // else no row of this warp exists
                    // the larger of both threads' values; each step comes here once, also after a
                    // wait that ran out, so that neither thread waits alone
                    auto both = [&](float best) {
                        s.best[t][team][row] = best;
                        asm volatile("bar.sync %0, 64;" ::"r"(4 + quarter) : "memory");
                        return fmaxf(best, s.best[t][team ^ 1][row]);
                    };
                    float f = 1.f;
                    if (!ok) {
                        both(-INFINITY);
                    } else {
                        const float *ks = s.ks[scs] + kHT * team, *vs = s.vs[scs] + kHT * team;
                        if (plain) {
                            f = soft_tile<!FOLD, false>(tS, ks, vs, a, ev, 0u, 0u, r, both);
                        } else {
                            uint32_t vis0 = 0, vis1 = 0;
                            const int wrow = w.mt * ROWS + blk + quarter * 32;
                            tree_visible(p, w.s, (wrow + lane) / p.group, wrow / p.group, min((wrow + 31) / p.group, w.s.n - 1), t0, valid, vis0, vis1);
                            if (unit.x != 0.f) f = soft_tile<!FOLD, true>(tS, ks, vs, a, ev, vis0, vis1, r, both);
                            else f = soft_exact(tS, ks, vs, a, vis0, vis1, r, both);
                        }
                        if (j >= 2 && __any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
                            for (int c = team * (D / 64); c < (team + 1) * (D / 64); ++c) {
                                uint32_t x[32];
                                tm_ld32(tO[0] + D * t + lanes + 32 * c, x);
                                tc_wait_ld32(x);
#pragma unroll
                                for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                                tm_st32(tO[0] + D * t + lanes + 32 * c, x);
                            }
                        }
                        tc_wait_st();
                    }
                }
                const SoftRow rt = r;
                r = r2;
                r2 = rt;
                const float ft = fac;
                fac = fac2;
                fac2 = ft;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    t_mbar_arrive(&s.p_full[t]);
                    if (NT == 1 || t == 1) t_mbar_arrive(&s.sc_empty[scs]);
                }
            }
            sc += T;
            if (J & 1) {
                const SoftRow rt = r;
                r = r2;
                r2 = rt;
            }

            // ---- the block's sums are complete ----
            const int brow = (NT == 2 ? team * 128 : 0) + row;               // row of the block
            const bool idle = (NT == 2 ? team * 128 : 0) + quarter * 32 >= rows;     // no row of this warp exists
            bool done = t_mbar_wait(&s.o_full[0], units & 1, &s.abort_flag, p.err);
            if (J > 1) done = t_mbar_wait(&s.o_full[1], units >> 1, &s.abort_flag, p.err) && done;
            units ^= J > 1 ? 3u : 1u;
            done = __all_sync(0xffffffffu, done);
            tc_fence_after();
            s.sum[team][0][row] = r.l;
            s.sum[team][1][row] = r2.l;
            both_sync();
            // reference and sum of a buffer's rows, and what becomes of them where nothing but NaN was seen
            auto settled = [&](int t, float M, float &l) {
                l = s.sum[0][t][row] + s.sum[1][t][row];
                M = M == -INFINITY && !(l == 0.f) ? 0.f : M;                   // any reference
                l = fminf(l, 3.4028234e38f) + (l != l ? l : 0.f);              // keeps NaN, bounds infinity
                return M;
            };
            float l, M, fa = 1.f, fb = 0.f;                                   // fa, fb: factors of the accumulators
            if constexpr (NT == 1) {
                float la, lb;
                const float ma = settled(0, r.M, la), mb = settled(1, r2.M, lb);
                M = fmaxf(ma, mb);
                fa = ma == -INFINITY ? 0.f : ex2(ma - M);
                fb = mb == -INFINITY ? 0.f : ex2(mb - M);
                l = la * fa + lb * fb;
            } else {
                M = settled(team, team ? r2.M : r.M, l);
            }
            const uint32_t oa = (NT == 2 ? tO[team] : tO[0]) + lanes, ob = tO[1] + lanes;
            const bool live = brow < rows && done;
            // the pieces before this one: fo times what lies in the slot
            const int64_t at_row = (int64_t)tree_slot(w, begin) * ROWS + brow;
            float *const part = p.part + at_row * D;
            float2 *const ml = reinterpret_cast<float2 *>(p.part + (int64_t)2 * p.ctas * ROWS * D) + at_row;
            float fo = 0.f;
            if (!w.begins && live) {
                const float2 x = *ml;
                if (x.x != -INFINITY) {
                    const float t = fmaxf(M, x.x), f = M == -INFINITY ? 0.f : ex2(M - t);
                    fo = ex2(x.x - t);
                    fa *= f;
                    fb *= f;
                    l = (f == 0.f ? 0.f : l * f) + x.y * fo;
                    M = t;
                }
            }
            if constexpr (NT == 1) {
                if (!w.begins) both_sync();           // both threads of a row have read its sum
            }
            // 32 accumulator columns, joined, in the order of the dims
            auto load32 = [&](int c, float (&v)[32]) {
                uint32_t x[32];
                tm_ld32(oa + 32 * c, x);
                tc_wait_ld32(x);
#pragma unroll
                for (int i = 0; i < 32; ++i) v[(i & ~7) + perm8(i & 7)] = fa == 0.f ? 0.f : __uint_as_float(x[i]) * fa;
                if constexpr (NT == 1) {
                    tm_ld32(ob + 32 * c, x);
                    tc_wait_ld32(x);
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (fb != 0.f) v[(i & ~7) + perm8(i & 7)] += __uint_as_float(x[i]) * fb;
                }
                if (fo != 0.f) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 y = *reinterpret_cast<const float4 *>(part + 32 * c + i);
                        v[i] += y.x * fo;
                        v[i + 1] += y.y * fo;
                        v[i + 2] += y.z * fo;
                        v[i + 3] += y.w * fo;
                    }
                }
            };
            constexpr int C0 = 1, STEP = NT == 2 ? 1 : 2;                     // NT = 1: the teams share the columns
            const int cfirst = NT == 2 ? 0 : team * C0;
            const int gr = w.mt * ROWS + brow;
            if (!w.whole) {
                if (!idle) {
#pragma unroll 1
                    for (int c = cfirst; c < D / 32; c += STEP) {
                        float v[32];
                        load32(c, v);
                        if (live) {
#pragma unroll
                            for (int i = 0; i < 32; i += 4)
                                *reinterpret_cast<float4 *>(part + 32 * c + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                        }
                    }
                }
                if (live && (NT == 2 || team == 0)) *ml = make_float2(M, l);
            } else {
                const float il = l == 0.f ? 0.f : 1.f / l;
                const bool turn = !(p.flags & RQ_ATTN_ROTATED_OUT);
                const int64_t o = ((w.s.row0 + gr / p.group) * p.kv_heads + w.h) * p.group + gr % p.group;
                char *dst = static_cast<char *>(p.out) + o * D * 2;
                // low 5 index bits of the butterflies, 32 columns at a time, back in place
                if (!idle) {
#pragma unroll 1
                    for (int c = cfirst; c < D / 32; c += STEP) {
                        float v[32];
                        load32(c, v);
                        if (turn) {
                            if (!signs_first) {
                                const uint32_t m = s.sign_words[c];
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] = (m >> i) & 1 ? -v[i] : v[i];
                            }
#pragma unroll
                            for (int st = 1; st < 32; st <<= 1)
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (!(i & st)) {
                                        const float x = v[i], y = v[i + st];
                                        v[i] = x + y;
                                        v[i + st] = x - y;
                                    }
                        }
                        uint32_t x[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(v[i]);
                        tm_st32(oa + 32 * c, x);
                    }
                    tc_wait_st();
                }
                if constexpr (NT == 1) {
                    tc_fence_before();
                    both_sync();
                    tc_fence_after();
                }
                // the upper bits, 8 columns of each 32 at a time, and out
                if (!idle) {
                    const float f = il * (turn ? inv_sqrt_dim<D>() : 1.f);
#pragma unroll 1
                    for (int g = cfirst; g < 4; g += STEP) {
                        uint32_t x[D / 32][8];
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) tm_ld8(oa + 32 * c + 8 * g, x[c]);
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) tc_wait_ld8(x[c]);
                        float v[D / 32][8];
#pragma unroll
                        for (int c = 0; c < D / 32; ++c)
#pragma unroll
                            for (int i = 0; i < 8; ++i) v[c][i] = __uint_as_float(x[c][i]);
                        if (turn) {
#pragma unroll
                            for (int st = 1; st < D / 32; st <<= 1)
#pragma unroll
                                for (int c = 0; c < D / 32; ++c)
                                    if (!(c & st)) {
#pragma unroll
                                        for (int i = 0; i < 8; ++i) {
                                            const float y = v[c][i], z = v[c + st][i];
                                            v[c][i] = y + z;
                                            v[c + st][i] = y - z;
                                        }
                                    }
                        }
#pragma unroll
                        for (int c = 0; c < D / 32; ++c) {
                            const uint32_t m = turn && signs_first ? s.sign_words[c] >> (8 * g) : 0u;
                            float y[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) y[i] = ((m >> i) & 1 ? -v[c][i] : v[c][i]) * f;
                            if (live) *reinterpret_cast<uint4 *>(dst + (32 * c + 8 * g) * 2) = pack16<IN>(y);
                        }
                    }
                }
            }
            tc_fence_before();
            if constexpr (NT == 1) both_sync();       // both accumulators are read: the next block may begin
            else team_sync();                         // s.work may be written again
        }
    } else if (warp >= 4 + kSoftWarps) {
        // ---------------- converters ----------------
        const int ct = threadIdx.x & (32 * kTeamWarps - 1);                  // thread of the team
        const uint32_t cteam = (warp - 4 - kSoftWarps) / kTeamWarps;
        // 16 bytes of codes: 32 dims of one token -> four 16-byte pieces of the operand.  A
        // warp loads 8 whole rows at a time; 8 lanes store 8 rows of one piece, so that no
        // two share a bank.  Thread: chunk ch of rows r0, r0 + RSTEP, ...
        constexpr int CH = RB / 16, N = kTcTT * CH / (32 * kTeamWarps), RSTEP = kTcTT / N;
        const int r0 = (ct & 7) | ((ct / (8 * CH)) << 3), ch = (ct >> 3) % CH;
        uint8_t *const dst0 = s.op[0] + (ch >> 1) * S::PANEL + r0 * 128;
        uint32_t piece[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) piece[q] = (uint32_t)(((ch & 1) * 4 + q) ^ (r0 & 7)) << 4;
        uint32_t base = 0, sc = 0;                       // items and tiles of earlier stretches
        for (int64_t at = begin; at < end;) {
            const TreeWork w = tree_work<ROWS, kTcTT>(p, s.line, at, begin, end);
            const int T = w.t1 - w.t0;
            at += w.used;
            if (T <= 0) continue;
            // a pipeline of three items: pages of the second next, codes and scales of the next
            int32_t pg[N];
            uint4 nx[N];
            float nf[N];
            auto pages = [&](int i) {
                int k;
                bool is_v;
                item_at<NT>(i, T, k, is_v);
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int t = (w.t0 + k) * kTcTT + r0 + n * RSTEP;
                    pg[n] = -1;
                    if (i < 2 * T && t < w.s.len) pg[n] = p.table[w.b * p.width + (t >> p.log_page)];
                }
            };
            auto load = [&](int i) {
                int k;
                bool is_v;
                item_at<NT>(i, T, k, is_v);
                const uint8_t *codes = (is_v ? p.vq : p.kq) + ch * 16;
                const float *scales = is_v ? p.vs : p.ks;
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    const int t = (w.t0 + k) * kTcTT + r0 + n * RSTEP;
                    nx[n] = make_uint4(0u, 0u, 0u, 0u);
                    nf[n] = 0.f;
                    if (pg[n] >= 0 && pg[n] < p.pages) {
                        const int64_t row = (((int64_t)pg[n] * p.kv_heads + w.h) << p.log_page) + (t & ((1 << p.log_page) - 1));
                        nx[n] = ld_once(codes + row * RB);
                        if (FOLD) nf[n] = scales[row];
                    }
                }
            };
            int i = (int)((cteam + kConvTeams - base % kConvTeams) % kConvTeams);       // this team's next item
            pages(i);
            load(i);
            pages(i + kConvTeams);
            for (; i < 2 * T; i += kConvTeams) {
                const uint32_t it = base + i, slot = it % kOps;
                int k;
                bool is_v;
                item_at<NT>(i, T, k, is_v);
                uint4 x[N];
                float f[N];
#pragma unroll
                for (int n = 0; n < N; ++n) {
                    x[n] = nx[n];
                    f[n] = nf[n];
                }
                load(i + kConvTeams);
                pages(i + 2 * kConvTeams);
                const uint32_t scs = (sc + k) % kSc;
                bool ok = warp_wait(&s.sc_full[scs], ((sc + k) / kSc) & 1, &s.abort_flag, p.err);
                ok = warp_wait(&s.op_empty[slot], ((it / kOps) & 1) ^ 1, &s.abort_flag, p.err) && ok;
                if (ok) {
                    const float2 unit = s.unit[scs];
                    const bool fold = FOLD && unit.x != 0.f;
                    const float down = !FOLD ? 1.f : is_v ? pow2(-(int)unit.y) : __uint_as_float((254u << 23) - __float_as_uint(unit.x));   // 1 / 2^ek
                    uint8_t *const dst = dst0 + slot * S::TILE;
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const uint32_t xw[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
                        const float fn = fold ? f[n] * down : 1.f;
                        const __half fh = __float2half_rn(fn);
                        const __half2 hi = __half2half2(fh), lo = __float2half2_rn(fn - __half2float(fh));
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *reinterpret_cast<uint4 *>(dst + n * RSTEP * 128 + piece[q]) = operands(xw[q], hi, lo);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    t_mbar_arrive(&s.op_full[slot]);
                    if (is_v) t_mbar_arrive(&s.sc_empty[scs]);
                }
            }
            base += 2 * T;
            sc += T;
        }
    }

    __syncwarp();
    // no MMA outlives the block, also when it gave up
    if (s.abort_flag) {
        const long long t0 = clock64();
        while (clock64() - t0 < 20000000ll) __nanosleep(1000);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

template <int IN, int D, int NT, int HV>
cudaError_t launch_tc(TreeParams &p, cudaStream_t stream) {
    auto kern = attn_tree_tc_kernel<IN, D, NT, HV>;
    const size_t smem = sizeof(TSmem<D, NT, HV>) + 1024;
    static_assert(sizeof(TSmem<D, NT, HV>) + 1024 <= 232448, "shared memory of one block");
    static std::atomic<uint64_t> allowed;
    cudaError_t e = allow_smem((const void *)kern, smem, allowed);
    if (e != cudaSuccess) return e;
    kern<<<p.ctas, kTcThreads, smem, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_tree_join<IN, D, 128 * NT>(p, stream);
}

}  // namespace

// Blocks of 128 rows pay a long start and end per unit, blocks of 16 rows more per token and
// row.  Measured (8 KV heads x 128, cold caches), here and there: 16 sequences of 4k, bf16,
// 32 rows 81 and 71 us, 48 rows 81 and 94, 64 rows 84 and 116; 64 of 300, 32 rows 66 and 63,
// 48 rows 68 and 84; fp16, 4 of 32k, 32 rows 120 and 115, 48 rows 122 and 161.  Where there
// are fewer tiles than SMs either does (2 of 512, 64 rows: 23 and 24).  The rows are those
// that there are on average, the tiles as many as the table can name.
bool attn_tree_tc_supported(const TreeCall &c) {
    const int64_t rows = tree_rows(c), tiles = tree_tiles(c, 128, kTcTT);
    return c.in_type != IN_F32 && (c.head_dim == 64 || c.head_dim == 128) && rows > 32 && tiles > device_sm_count();
}

int64_t attn_tree_tc_workspace(int64_t head_dim) {
    if (head_dim != 64 && head_dim != 128) return 0;
    const int sms = device_sm_count();
    return tree_join_at(sms, 256, (int)head_dim) * (int64_t)sizeof(float) + sms * (int64_t)sizeof(TreeJoin);
}

cudaError_t launch_attn_tree_tc(const TreeCall &c, cudaStream_t stream) {
    TreeParams p;
    if (!tree_params(c, p)) return cudaErrorUnknown;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorUnknown;
    // two row blocks share each converted tile; fp16 queries keep the second's shared
    // memory for the low parts of q~
    const int nt = tree_rows(c) > 128 && c.in_type == IN_BF16 ? 2 : 1;
    tree_ctas(c, p, 128 * nt, kTcTT, sms);
    const bool d128 = c.head_dim == 128;
    if (c.in_type == IN_F16)
        return d128 ? launch_tc<IN_F16, 128, 1, 2>(p, stream) : launch_tc<IN_F16, 64, 1, 2>(p, stream);
    if (nt == 2)
        return d128 ? launch_tc<IN_BF16, 128, 2, 1>(p, stream) : launch_tc<IN_BF16, 64, 2, 1>(p, stream);
    return d128 ? launch_tc<IN_BF16, 128, 1, 1>(p, stream) : launch_tc<IN_BF16, 64, 1, 1>(p, stream);
}

}  // namespace rq
