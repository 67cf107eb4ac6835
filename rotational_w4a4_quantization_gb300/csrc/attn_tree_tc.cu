// attn_tree_tc.cu -- tree attention over the paged rotated INT4 cache on the
// 5th-generation tensor cores (sm_103a): blocks of 128 or 256 query rows.
//
// The same operator as attn_tree.cu (see there for the formulas).  Here the rows
// (nodes x query heads of a KV head) fill the 128 lanes of a tcgen05 MMA:
//   S = Q K^T   M128 N128 (tokens) K = D,  A = q~ in shared memory, fp16
//   O += P V    M128 N = D  K128 (tokens), A = P in tensor memory, fp16
// and a tile is 128 tokens.  Two softmax teams of 128 threads (one row each) work in
// turn with the tensor core: while it runs P V and the next Q K^T for one team, the
// other team turns its scores into weights.
//   NT = 2: 256 rows, team w has rows 128 w ..; every tile is used by both.
//   NT = 1: 128 rows; team w takes the tiles of parity w with an accumulator of its
//           own, and the two are joined at the end.
//
// Roles (16 warps, one block per SM):
//   warp 0       TMA: packed code tiles (8 KB each at D = 128) and scales
//   warp 1       tensor memory, all MMAs (one lane)
//   warps 4-11   softmax teams
//   warps 12-15  converters: packed codes -> fp16 codes (exact) in the 128-byte-
//                swizzled operand layout.  One layout serves both products: rows of
//                64 dims per token are K-major for Q K^T and MN-major for P V.
// Tensor memory, 512 columns: S0 S1 (128 each; P overwrites the first half of its S)
// and O0 O1 (D each).
//
// Weights: w = 2^(s - M) vs is what the MMA sees, rounded to fp16; the sum l adds
// 2^(s - M) in fp32.  O / l does not depend on M, so M only has to keep w in range: it
// follows the largest s + log2 vs, and moves only when some w passes 2^8 (the
// accumulator is then rescaled in place, between the commit that delivers S and the
// arrival that delivers P, when no MMA touches it).
// The scales of K stay out of the product: s = (q~ . code) ks in fp32.
// fp16 queries: q~ carries 22 bits (two fp16 parts, Q K^T twice), as their outputs
// resolve the rounding of q~ to 11 bits.
#include "rq.h"
#include "rq_internal.h"
#include "tree_device.cuh"

namespace rq {
namespace {

constexpr int kTcTT = 128;               // tokens per tile
constexpr int kOps = 3;                  // operand slots
constexpr int kSc = 4;                   // scale slots
constexpr int kSoftWarps = 8, kConvWarps = 4;
constexpr int kTcThreads = 32 * (4 + kSoftWarps + kConvWarps);

template <int D, int NT, int HV>
struct TSmem {
    static constexpr int RB = D / 2;                        // packed bytes of a token
    static constexpr int RAW = NT * HV == 2 ? 6 : 8;        // packed tiles in flight
    static constexpr int PANEL = 128 * 128;                 // 128 rows x 64 dims of fp16
    static constexpr int TILE = D / 64 * PANEL;
    alignas(1024) uint8_t q[NT * HV][TILE];
    alignas(1024) uint8_t op[kOps][TILE];
    alignas(1024) uint8_t rawt[RAW][kTcTT * RB];
    alignas(16) float ks[kSc][kTcTT];
    alignas(16) float vs[kSc][kTcTT];
    float2 rfac[NT * 128];                                  // a row's factors: s = (a S + b) ks
    float ref[2][128], sum[2][128];                         // NT = 1: the teams' references and sums
    int64_t prefix[kScan + 1];
    alignas(8) uint64_t raw_full[RAW], raw_empty[RAW];
    uint64_t sc_full[kSc], sc_empty[kSc];
    uint64_t op_full[kOps], op_empty[kOps];
    uint64_t q_full, s_full[2], p_full[2], o_full[2];
    uint32_t valid[kSc];
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
__device__ __forceinline__ void tm_st16(uint32_t t, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
                 RQ_W8(r, 0), RQ_W8(r, 8) : "memory");
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

// A word of 8 codes as 8 fp16 operands, in the order of the dims 0 4 1 5 2 6 3 7.
// Values: 0x6400 | u is 1024 + u, so nibbles 0 and 4 (u = code + 8 after the sign bit's
// flip) lose 1032, nibbles 1 and 5, which stay four bits up, are 1024 + 16 u: times
// 1/16, less 72.  Exact.
__device__ __forceinline__ uint4 v_operands(uint32_t x) {
    const __half2 m0 = __half2half2(__ushort_as_half(0xe408)), r16 = __half2half2(__ushort_as_half(0x2c00)),
                  m1 = __half2half2(__ushort_as_half(0xd480));             // -1032, 1/16, -72
    uint32_t r[4];
#pragma unroll
    for (int j = 0; j < 4; j += 2) {
        const uint32_t y = x >> (4 * j);
        const uint32_t a = (y & 0x000f000fu) ^ 0x64086408u, b = (y & 0x00f000f0u) ^ 0x64806480u;
        const __half2 ha = __hadd2(*reinterpret_cast<const __half2 *>(&a), m0);
        const __half2 hb = __hfma2(*reinterpret_cast<const __half2 *>(&b), r16, m1);
        r[j] = *reinterpret_cast<const uint32_t *>(&ha);
        r[j + 1] = *reinterpret_cast<const uint32_t *>(&hb);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}
// Keys: no arithmetic.  u = code + 8 as the subnormal u 2^-24 (nibbles 1, 3, 5, 7:
// 16 u 2^-24, and q~ holds a sixteenth there); the softmax takes 2^24 and 8 sum q~ out
// again with the row's factors.  The sums are short (D terms), so nothing is lost.
__device__ __forceinline__ uint4 k_operands(uint32_t x) {
    const uint32_t y = x >> 8;
    return make_uint4((x ^ 0x00080008u) & 0x000f000fu, (x ^ 0x00800080u) & 0x00f000f0u,
                      (y ^ 0x00080008u) & 0x000f000fu, (y ^ 0x00800080u) & 0x00f000f0u);
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
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

// Which of the tokens t .. t + 15 (rows at .. of a tile with page pieces `valid`) a node
// sees, as bits.  The mask bytes are loaded all at once.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : (n >= 16 ? 0xffffu : (1u << n) - 1u); }
__device__ __forceinline__ uint32_t tree_visible(const TreeParams &p, const TreeWork &w, int node, int t, int at, uint32_t valid) {
    if (node >= w.s.n || !((valid >> (at >> min(p.log_page, 7))) & 1)) return 0u;
    const uint32_t there = below(w.s.len - t);
    const int j0 = t - w.s.ctx;                                   // the node at token t
    if (!p.mask) return there & below(node + 1 - j0);
    uint32_t seen = below(-j0);
    if (j0 + 16 > 0 && j0 < w.s.n) {
        const uint8_t *m = p.mask + (w.s.row0 + node) * p.mask_stride + j0;
        uint8_t x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = (unsigned)(j0 + i) < (unsigned)w.s.n ? m[i] : (uint8_t)0;
#pragma unroll
        for (int i = 0; i < 16; ++i) seen |= x[i] ? 1u << i : 0u;
    }
    return there & seen;
}

constexpr int kCW = 16;                  // scores that a row works on at a time: more of them spill

// A row's kCW raw scores -> s - M, with s = (a S + b) ks.
__device__ __forceinline__ void soft_scores(const uint32_t (&sr)[kCW], const float *ks, float2 fac, float M,
                                            float2 (&t)[kCW / 2]) {
    const float2 a2 = make_float2(fac.x, fac.x), b2 = make_float2(fac.y, fac.y), nm = make_float2(-M, -M);
    const float4 *k4 = reinterpret_cast<const float4 *>(ks);
#pragma unroll
    for (int i = 0; i < kCW / 4; ++i) {
        const float4 k = k4[i];
        const float2 x = make_float2(__uint_as_float(sr[4 * i]), __uint_as_float(sr[4 * i + 1]));
        const float2 y = make_float2(__uint_as_float(sr[4 * i + 2]), __uint_as_float(sr[4 * i + 3]));
        t[2 * i] = __ffma2_rn(__ffma2_rn(x, a2, b2), make_float2(k.x, k.y), nm);
        t[2 * i + 1] = __ffma2_rn(__ffma2_rn(y, a2, b2), make_float2(k.z, k.w), nm);
    }
}
// Weights of kCW scores: p = 2^t (their sum is returned), w = p vs as fp16 pairs.
__device__ __forceinline__ float soft_weights(const float2 (&t)[kCW / 2], const float *vs, uint32_t (&pk)[kCW / 2]) {
    const float4 *v4 = reinterpret_cast<const float4 *>(vs);
    float2 sum[2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll
    for (int i = 0; i < kCW / 4; ++i) {
        const float4 v = v4[i];
        const float2 p0 = make_float2(ex2(t[2 * i].x), ex2(t[2 * i].y));
        const float2 p1 = make_float2(ex2(t[2 * i + 1].x), ex2(t[2 * i + 1].y));
        sum[0] = __fadd2_rn(sum[0], p0);
        sum[1] = __fadd2_rn(sum[1], p1);
        const float2 w0 = __fmul2_rn(p0, make_float2(v.x, v.y)), w1 = __fmul2_rn(p1, make_float2(v.z, v.w));
        const __half2 h0 = __floats2half2_rn(w0.x, w0.y), h1 = __floats2half2_rn(w1.x, w1.y);
        pk[2 * i] = *reinterpret_cast<const uint32_t *>(&h0);
        pk[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&h1);
    }
    const float2 s2 = __fadd2_rn(sum[0], sum[1]);
    return s2.x + s2.y;
}

// One row's state: the reference M (-inf: nothing seen yet), the sum l, and the factor
// F that the sums of earlier tiles still need.
struct SoftRow {
    float M, l, F;
};

// Chunk c of a tile with everything that is rare: masks (the low bits of `vis` name the
// visible tokens), the first reference, a reference that has to move.  A masked weight
// is zero whatever the value's scale holds.  The chunk's scores lie in tensor memory,
// the tile's earlier weights over the scores before them.
__device__ __forceinline__ void soft_careful(uint32_t tS, int c, const float *ks, const float *vs, float2 fac, uint32_t vis,
                                             SoftRow &r) {
    uint32_t sr[kCW];
    float2 t[kCW / 2];
    tm_ld16(tS + kCW * c, sr);
    tc_wait_ld16(sr);
    soft_scores(sr, ks, fac, r.M == -INFINITY ? 0.f : r.M, t);
    float cand = -INFINITY, tmax = -INFINITY;                     // log2 of the largest w and p, against M
#pragma unroll
    for (int i = 0; i < kCW / 2; ++i) {
        const float2 v = reinterpret_cast<const float2 *>(vs)[i];
        const bool s0 = (vis >> (2 * i)) & 1, s1 = (vis >> (2 * i + 1)) & 1;
        t[i] = make_float2(s0 ? t[i].x : -INFINITY, s1 ? t[i].y : -INFINITY);
        if (s0) cand = fmaxf(cand, t[i].x + lg2(v.x));
        if (s1) cand = fmaxf(cand, t[i].y + lg2(v.y));
        tmax = max3(tmax, t[i].x, t[i].y);
    }
    cand = fmaxf(cand, tmax - 100.f);                             // rows of zero values: keeps p itself finite
    float up = 0.f, f = 1.f;
    if (r.M == -INFINITY) {
        if (vis) r.M = up = cand == -INFINITY ? 0.f : cand;       // nothing but NaN seen: any reference
    } else if (cand > 8.f) {
        up = cand;
        f = ex2(-up);
        r.M += up;
        r.l *= f;
        r.F *= f;
    }
    if (__any_sync(0xffffffffu, f != 1.f)) {
        const __half2 fh = __half2half2(__float2half_rn(f));
        for (int cc = 0; cc < c; ++cc) {                          // this tile's earlier weights
            uint32_t x[8];
            tm_ld8(tS + kCW / 2 * cc, x);
            tc_wait_ld8(x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const __half2 y = __hmul2(*reinterpret_cast<const __half2 *>(&x[i]), fh);
                x[i] = *reinterpret_cast<const uint32_t *>(&y);
            }
            tm_st8(tS + kCW / 2 * cc, x);
        }
        tc_wait_st();
    }
#pragma unroll
    for (int i = 0; i < kCW / 2; ++i) t[i] = make_float2(t[i].x - up, t[i].y - up);
    uint32_t pk[kCW / 2];
    r.l += soft_weights(t, vs, pk);
#pragma unroll
    for (int i = 0; i < kCW / 2; ++i)
        pk[i] &= ((vis >> (2 * i)) & 1 ? 0x0000ffffu : 0u) | ((vis >> (2 * i + 1)) & 1 ? 0xffff0000u : 0u);
    tm_st8(tS + kCW / 2 * c, pk);
}

// One row's 128 scores of a tile that every row sees whole; the next kCW are on their
// way while these are worked on.  Whether a weight leaves fp16's range is seen from the
// sum of kCW p (needed anyway) times their largest vs: it is at most kCW times the
// largest w, so below 2^13 all is well, and only a w above 2^9 can pass that.  Returns
// the number of chunks done: the rest, from the first that is not well, need care.
__device__ __forceinline__ int soft_tile(uint32_t tS, const float *ks, const float *vs, float2 fac, SoftRow &r) {
    uint32_t sr[2][kCW];
    tm_ld16(tS, sr[0]);
    const float4 v = reinterpret_cast<const float4 *>(vs)[threadIdx.x & 31];
    float vtop = fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w));         // each kCW / 4 lanes: a chunk's largest vs
#pragma unroll
    for (int o = 1; o < kCW / 4; o <<= 1) vtop = fmaxf(vtop, __shfl_xor_sync(0xffffffffu, vtop, o));
#pragma unroll
    for (int c = 0; c < kTcTT / kCW; ++c) {
        const float vmax = __shfl_sync(0xffffffffu, vtop, kCW / 4 * c);
        float2 t[kCW / 2];
        tc_wait_ld16(sr[c & 1]);
        // the next columns are overwritten after chunk 2 c + 1 at the earliest
        if (c + 1 < kTcTT / kCW) tm_ld16(tS + kCW * (c + 1), sr[(c + 1) & 1]);
        soft_scores(sr[c & 1], ks + kCW * c, fac, r.M, t);
        uint32_t pk[kCW / 2];
        const float add = soft_weights(t, vs + kCW * c, pk);
        // also where r.M = -inf: add is infinite or NaN
        if (__any_sync(0xffffffffu, !(add * vmax <= 8192.f && add <= 1e30f))) return c;
        r.l += add;
        tm_st8(tS + kCW / 2 * c, pk);
    }
    return kTcTT / kCW;
}

template <int IN, int D, int NT, int HV>
__global__ void __launch_bounds__(kTcThreads, 1)
attn_tree_tc_kernel(const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv,
                    const __grid_constant__ TreeParams p) {
    using S = TSmem<D, NT, HV>;
    constexpr int ROWS = 128 * NT, RB = D / 2, RAW = S::RAW, E = D / 32;
    extern __shared__ uint8_t raw[];
    S &s = *reinterpret_cast<S *>(raw + ((1024u - (t_smem(raw) & 1023u)) & 1023u));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < RAW; ++i) {
            t_mbar_init(&s.raw_full[i], 1);
            t_mbar_init(&s.raw_empty[i], kConvWarps);
        }
        for (int i = 0; i < kSc; ++i) {
            t_mbar_init(&s.sc_full[i], 1);
            t_mbar_init(&s.sc_empty[i], 4 * NT);
        }
        for (int i = 0; i < kOps; ++i) {
            t_mbar_init(&s.op_full[i], kConvWarps);
            t_mbar_init(&s.op_empty[i], 1);
        }
        t_mbar_init(&s.q_full, kSoftWarps);
        for (int i = 0; i < 2; ++i) {
            t_mbar_init(&s.s_full[i], 1);
            t_mbar_init(&s.p_full[i], 4);
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
    tc_fence_before();
    tree_scan<ROWS, kTcTT>(p, s.prefix);               // ends with a block barrier
    tc_fence_after();
    const uint32_t tmem = s.tmem_base;
    const uint32_t tS[2] = {tmem, tmem + 128}, tO[2] = {tmem + 256, tmem + 256 + (uint32_t)D};
    const int64_t total = s.prefix[kScan];
    const int64_t begin = tree_begin(total, p.ctas, blockIdx.x), end = tree_begin(total, p.ctas, blockIdx.x + 1);

    if (warp == 0) {
        // ---------------- producer ----------------
        const int bt = min(kTcTT, 1 << p.log_page), pieces = kTcTT / bt;
        uint32_t it = 0, sc = 0;                       // items and tiles so far
        for (int64_t at = begin; at < end;) {
            const TreeWork w = tree_work<ROWS, kTcTT>(p, s.prefix, at, end);
            const int T = w.t1 - w.t0;
            at += T;
            for (int i = 0; i < 2 * T; ++i, ++it) {
                int k;
                bool is_v;
                item_at<NT>(i, T, k, is_v);
                const int t = (w.t0 + k) * kTcTT + lane * bt;
                int64_t pg = -1;
                if (lane < pieces && t < w.s.len) {
                    pg = p.table[w.b * p.width + (t >> p.log_page)];
                    if (pg >= p.pages) pg = -1;
                }
                const int st = it % RAW;
                bool go = t_mbar_wait(&s.raw_empty[st], ((it / RAW) & 1) ^ 1, &s.abort_flag, p.err);
                const uint32_t scs = (sc + k) % kSc;
                if (!is_v) go &= t_mbar_wait(&s.sc_empty[scs], (((sc + k) / kSc) & 1) ^ 1, &s.abort_flag, p.err);
                const uint32_t valid = __ballot_sync(0xffffffffu, pg >= 0 && go);
                if (lane == 0) {
                    t_mbar_expect(&s.raw_full[st], __popc(valid) * bt * RB);
                    if (!is_v) {
                        s.valid[scs] = valid;
                        t_mbar_expect(&s.sc_full[scs], __popc(valid) * bt * 8);
                    }
                }
                __syncwarp();
                if ((valid >> lane) & 1) {
                    const int64_t row = ((pg * p.kv_heads + w.h) << p.log_page) + (t & ((1 << p.log_page) - 1));
                    t_tma_2d(s.rawt[st] + lane * bt * RB, is_v ? &tmv : &tmk, &s.raw_full[st], (int)row);
                    if (!is_v) {
                        t_bulk(&s.ks[scs][lane * bt], p.ks + row, bt * 4, &s.sc_full[scs]);
                        t_bulk(&s.vs[scs][lane * bt], p.vs + row, bt * 4, &s.sc_full[scs]);
                    }
                }
            }
            sc += T;
        }
    } else if (warp == 1) {
        // ---------------- MMA ----------------
        // The whole warp runs the loop, so that descriptors stay in uniform registers;
        // one lane issues (16 MMAs of 64 cycles each per tile leave no time for more).
        const bool one = elect_one();
        uint32_t base = 0, unit = 0, pc[2] = {0, 0};         // items of earlier stretches; stretches; P tiles per team
        constexpr uint32_t id_qk = idesc_f16(kTcTT, false), id_pv = idesc_f16(D, true);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dq = op_desc(t_smem(s.q[0]), 16), dk = op_desc(t_smem(s.op[0]), 16);
        const uint64_t dv = op_desc(t_smem(s.op[0]), S::PANEL);
        bool ok = true;
        for (int64_t at = begin; at < end && ok; ++unit) {
            const TreeWork w = tree_work<ROWS, kTcTT>(p, s.prefix, at, end);
            const int T = __shfl_sync(0xffffffffu, w.t1 - w.t0, 0), J = NT * T;
            at += T;
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
                        mma_ts(tm + 256 + D * t, tm + 128 * t + 8 * c, b + c * (2048 >> 4), id_pv, j >= 2 || c > 0);
                    if (NT == 1 || t == 1) tc_commit(&s.op_empty[slot]);
                    if (j + 2 >= J) tc_commit(&s.o_full[t]);
                }
                __syncwarp();
                if (j + 2 < J) qk(j + 2);
            }
            base += 2 * T;
        }
    } else if (warp >= 4 && warp < 4 + kSoftWarps) {
        // ---------------- softmax teams ----------------
        const int team = (warp - 4) >> 2, quarter = warp & 3, row = quarter * 32 + lane;     // row of the 128
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        auto both_sync = [] { asm volatile("bar.sync 1, 256;" ::: "memory"); };
        const bool signs_first = (p.flags & RQ_SIGNS_FIRST) != 0;
        uint32_t sc = 0, uses = 0, units = 0;          // tiles so far; S tiles of this team; finished stretches of this team
        for (int64_t at = begin; at < end;) {
            const TreeWork w = tree_work<ROWS, kTcTT>(p, s.prefix, at, end);
            const int T = w.t1 - w.t0;
            at += T;
            const int rows = min(ROWS, w.s.n * p.group - w.mt * ROWS);        // of the block

            // ---- q~: each warp 32 (NT = 2) or 16 rows of the block's ----
            {
                constexpr int RW = ROWS / kSoftWarps, U = 8;         // U rows in flight
                float sg[E];
                lane_signs<E>(sg, lane, p.seed);
#pragma unroll 1
                for (int i = 0; i < RW; i += U) {
                    const int r0 = (warp - 4) * RW + i;
                    float v[U][E], top[U], sum[U];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int gr = w.mt * ROWS + r0 + u;
                        const char *src = static_cast<const char *>(p.q) +
                                          ((w.s.row0 + gr / p.group) * p.q_token + (w.h * p.group + gr % p.group) * p.q_head) * 2;
#pragma unroll
                        for (int e = 0; e < E; ++e) v[u][e] = r0 + u < rows ? load_elem<IN>(src, lane * E + e) : 0.f;
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        warp_rotate<E>(v[u], sg, lane, signs_first, inv_sqrt_dim<D>());
                        top[u] = 0.f;
#pragma unroll
                        for (int e = 0; e < E; ++e) top[u] = fmaxf(top[u], fabsf(v[u][e]));
                    }
#pragma unroll
                    for (int o = 16; o; o >>= 1)
#pragma unroll
                        for (int u = 0; u < U; ++u) top[u] = fmaxf(top[u], __shfl_xor_sync(0xffffffffu, top[u], o));
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const int r = r0 + u, rr = r & 127;
                        int ex = (int)((__float_as_uint(top[u]) >> 23) & 255u) - 126;      // top < 2^ex
                        ex = max(-100, min(ex, 104));
                        top[u] = __uint_as_float((uint32_t)(127 + ex) << 23) * p.score_scale;
                        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
                        sum[u] = 0.f;
#pragma unroll
                        for (int e = 0; e < E; ++e) {
                            const int d = lane * E + e;
                            const int pos = ((d & 3) << 1) + ((d >> 2) & 1);
                            const uint32_t off = (uint32_t)((d >> 6) * S::PANEL + rr * 128 + ((((d & 63) >> 3) ^ (rr & 7)) << 4) + pos * 2);
                            const float x = v[u][e] * down * (d & 1 ? 0.0625f : 1.f);
                            const __half hi = __float2half_rn(x);
                            float got = __half2float(hi);
                            *reinterpret_cast<__half *>(s.q[NT == 2 ? r >> 7 : 0] + off) = hi;
                            if constexpr (HV == 2) {
                                const __half lo = __float2half_rn(x - got);
                                got += __half2float(lo);
                                *reinterpret_cast<__half *>(s.q[1] + off) = lo;
                            }
                            sum[u] += got * (d & 1 ? 16.f : 1.f);
                        }
                    }
#pragma unroll
                    for (int o = 16; o; o >>= 1)
#pragma unroll
                        for (int u = 0; u < U; ++u) sum[u] += __shfl_xor_sync(0xffffffffu, sum[u], o);
                    if (lane == 0) {
#pragma unroll
                        for (int u = 0; u < U; ++u) s.rfac[r0 + u] = make_float2(top[u] * 16777216.f, -8.f * sum[u] * top[u]);
                    }
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) t_mbar_arrive(&s.q_full);
            both_sync();
            const int brow = (NT == 2 ? team * 128 : 0) + row;               // row of the block
            const float2 fac = s.rfac[brow];
            const bool idle = (NT == 2 ? team * 128 : 0) + quarter * 32 >= rows;     // no row of this warp exists
            const int node = (w.mt * ROWS + brow) / p.group;
            const uint32_t all = (uint32_t)((1ull << (kTcTT / min(kTcTT, 1 << p.log_page))) - 1);
            SoftRow r{-INFINITY, 0.f, 1.f};
            bool first = true;
            for (int k = NT == 2 ? 0 : team; k < T; k += NT == 2 ? 1 : 2, ++uses) {
                const uint32_t scs = (sc + k) % kSc;
                bool ok = t_mbar_wait(&s.sc_full[scs], ((sc + k) / kSc) & 1, &s.abort_flag, p.err);
                ok = t_mbar_wait(&s.s_full[team], uses & 1, &s.abort_flag, p.err) && ok;
                ok = __all_sync(0xffffffffu, ok);
                tc_fence_after();
                if (ok && !idle) {
                    const int t0 = (w.t0 + k) * kTcTT;
                    const uint32_t valid = s.valid[scs];
                    const bool masked = t0 + kTcTT > w.s.ctx || valid != all;
                    r.F = 1.f;
                    const int fast = masked ? 0 : soft_tile(tS[team] + lanes, s.ks[scs], s.vs[scs], fac, r);
#pragma unroll 1
                    for (int c = fast; c < kTcTT / kCW; ++c) {
                        const uint32_t vis = masked ? tree_visible(p, w, node, t0 + kCW * c, kCW * c, valid) : 0xffffu;
                        soft_careful(tS[team] + lanes, c, s.ks[scs] + kCW * c, s.vs[scs] + kCW * c, fac, vis, r);
                    }
                    if (!first && __any_sync(0xffffffffu, r.F != 1.f)) {
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            uint32_t x[32];
                            tm_ld32(tO[team] + lanes + 32 * c, x);
                            tc_wait_ld32(x);
#pragma unroll
                            for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * r.F);
                            tm_st32(tO[team] + lanes + 32 * c, x);
                        }
                    }
                    tc_wait_st();
                }
                first = false;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    t_mbar_arrive(&s.p_full[team]);
                    t_mbar_arrive(&s.sc_empty[scs]);
                }
            }
            sc += T;

            // ---- the block's sums are complete ----
            bool done = true;
            if (!first) {
                done = __all_sync(0xffffffffu, t_mbar_wait(&s.o_full[team], units & 1, &s.abort_flag, p.err));
                ++units;
            }
            tc_fence_after();
            float M = r.M, l = r.l;
            l = fminf(l, 3.4028234e38f) + (l != l ? l : 0.f);                 // keeps NaN, bounds infinity
            float fa = 1.f, fb = 0.f;                                         // factors of the teams' accumulators
            if constexpr (NT == 1) {
                s.ref[team][row] = M;
                s.sum[team][row] = l;
                both_sync();
                const float ma = s.ref[0][row], mb = s.ref[1][row];
                M = fmaxf(ma, mb);
                fa = ma == -INFINITY ? 0.f : ex2(ma - M);
                fb = mb == -INFINITY ? 0.f : ex2(mb - M);
                l = s.sum[0][row] * fa + s.sum[1][row] * fb;
            }
            const uint32_t oa = (NT == 2 ? tO[team] : tO[0]) + lanes, ob = tO[1] + lanes;
            const bool live = brow < rows && done;
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
            };
            constexpr int C0 = 1, STEP = NT == 2 ? 1 : 2;                     // NT = 1: the teams share the columns
            const int cfirst = NT == 2 ? 0 : team * C0;
            const int gr = w.mt * ROWS + brow;
            if (!w.whole) {
                const int64_t slot = 2 * (int64_t)blockIdx.x + (at - T == begin ? 0 : 1);
                float *part = p.part + (slot * ROWS + brow) * D;
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
                if (live && (NT == 2 || team == 0))
                    *reinterpret_cast<float2 *>(p.part + (int64_t)2 * p.ctas * ROWS * D + (slot * ROWS + brow) * 2) = make_float2(M, l);
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
        }
    } else if (warp >= 4 + kSoftWarps) {
        // ---------------- converters ----------------
        const int ct = threadIdx.x - 32 * (4 + kSoftWarps);                  // 0 .. 127
        uint32_t it = 0;
        for (int64_t at = begin; at < end;) {
            const TreeWork w = tree_work<ROWS, kTcTT>(p, s.prefix, at, end);
            const int T = w.t1 - w.t0;
            at += T;
            for (int i = 0; i < 2 * T; ++i, ++it) {
                const int st = it % RAW, slot = it % kOps;
                int k;
                bool is_v;
                item_at<NT>(i, T, k, is_v);
                bool ok = t_mbar_wait(&s.raw_full[st], (it / RAW) & 1, &s.abort_flag, p.err);
                ok = t_mbar_wait(&s.op_empty[slot], ((it / kOps) & 1) ^ 1, &s.abort_flag, p.err) && ok;
                if (ok) {
                    // 16 bytes of codes: 32 dims of one token -> four 16-byte pieces of the operand.
                    // 8 lanes take 8 rows of one chunk: no bank conflicts on either side.
                    constexpr int CH = RB / 16, N = kTcTT * CH / (32 * kConvWarps);
                    uint4 x[N];
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const int u = ct + n * 32 * kConvWarps;
                        const int r = (u & 7) | ((u / (8 * CH)) << 3), ch = (u >> 3) % CH;
                        const int sw = CH == 4 ? ch ^ ((r >> 1) & 3) : ch ^ ((r >> 2) & 1);
                        x[n] = *reinterpret_cast<const uint4 *>(s.rawt[st] + r * RB + sw * 16);
                    }
#pragma unroll
                    for (int n = 0; n < N; ++n) {
                        const int u = ct + n * 32 * kConvWarps;
                        const int r = (u & 7) | ((u / (8 * CH)) << 3), ch = (u >> 3) % CH;
                        const uint32_t xw[4] = {x[n].x, x[n].y, x[n].z, x[n].w};
                        uint8_t *dst = s.op[slot] + (ch >> 1) * S::PANEL + r * 128;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            *reinterpret_cast<uint4 *>(dst + ((((ch & 1) * 4 + q) ^ (r & 7)) << 4)) =
                                is_v ? v_operands(xw[q]) : k_operands(xw[q]);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    t_mbar_arrive(&s.op_full[slot]);
                    t_mbar_arrive(&s.raw_empty[st]);
                }
            }
        }
    }

    __syncwarp();
    // no copy and no MMA outlives the block, also when it gave up
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
cudaError_t launch_tc(TreeParams &p, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t stream) {
    auto kern = attn_tree_tc_kernel<IN, D, NT, HV>;
    const size_t smem = sizeof(TSmem<D, NT, HV>) + 1024;
    static_assert(sizeof(TSmem<D, NT, HV>) + 1024 <= 232448, "shared memory of one block");
    static std::atomic<uint64_t> allowed;
    cudaError_t e = allow_smem((const void *)kern, smem, allowed);
    if (e != cudaSuccess) return e;
    kern<<<p.ctas, kTcThreads, smem, stream>>>(mk, mv, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int bph = (int)(((int64_t)p.max_nodes * p.group + 128 * NT - 1) / (128 * NT));
    const int64_t units = (int64_t)p.seqs * p.kv_heads * bph;
    if (units > 0x7fffffffll) return cudaErrorInvalidValue;
    attn_tree_join_kernel<IN, D, 128 * NT, kTcTT>
        <<<dim3((unsigned)units, 128 * NT / kJoinWarps), 32 * kJoinWarps, 0, stream>>>(p, bph);
    return cudaGetLastError();
}

}  // namespace

bool attn_tree_tc_supported(int in_type, int64_t head_dim, int64_t rows) {
    return in_type != IN_F32 && (head_dim == 64 || head_dim == 128) && rows > 16;
}

int64_t attn_tree_tc_workspace(int64_t head_dim) {
    return 2 * (int64_t)device_sm_count() * 256 * (head_dim + 2) * (int64_t)sizeof(float);
}

cudaError_t launch_attn_tree_tc(const TreeCall &c, cudaStream_t stream) {
    TreeParams p;
    if (!tree_params(c, p)) return cudaErrorUnknown;
    const int sms = device_sm_count();
    if (sms <= 0) return cudaErrorUnknown;
    const int64_t rows = c.max_nodes * p.group;
    // two row blocks share each converted tile; fp16 queries keep the second's shared
    // memory for the low parts of q~
    const int nt = rows > 128 && c.in_type == IN_BF16 ? 2 : 1;
    const int64_t bph = (rows + 128 * nt - 1) / (128 * nt);
    const int64_t max_tiles = c.seqs * c.cache.heads * bph * ((c.width * c.cache.page_size + kTcTT - 1) / kTcTT);
    p.ctas = (int)(max_tiles < sms ? max_tiles : sms);
    CUtensorMap mk, mv;
    if (!tree_maps(c, kTcTT, mk, mv)) return cudaErrorInvalidValue;
    const bool d128 = c.head_dim == 128;
    if (c.in_type == IN_F16)
        return d128 ? launch_tc<IN_F16, 128, 1, 2>(p, mk, mv, stream) : launch_tc<IN_F16, 64, 1, 2>(p, mk, mv, stream);
    if (nt == 2)
        return d128 ? launch_tc<IN_BF16, 128, 2, 1>(p, mk, mv, stream) : launch_tc<IN_BF16, 64, 2, 1>(p, mk, mv, stream);
    return d128 ? launch_tc<IN_BF16, 128, 1, 1>(p, mk, mv, stream) : launch_tc<IN_BF16, 64, 1, 1>(p, mk, mv, stream);
}

}  // namespace rq
