// kv_paged.cu -- the paged rotated INT4 KV cache: quantising rows as they are
// written to their slots, and reading sequences back dense (sm_103a).
//
// "End-to-end flow" (The KV cache) of the QuaRot page: keys (after their rotary
// positions) and values are rotated head by head and stored in four bits.
//   write: y = x R, scale = max|y| / 7, code = round_half_even(y / scale)
//   read:  x^ = (code * scale) R^T, or code * scale where the rotated basis is kept
// A page holds page_size tokens of every head, head-major: codes
// [page][head][row][D/2], scales [page][head][row].
//
// Both are bound by moving the rows once (D elements on one side, D/2 + 4 bytes on
// the other).  A row is spread over 4 lanes (8 for D = 256), 32 elements each at
// D = 128, interleaved in 8-element chunks so that every load and store covers whole
// lines: 5 of the 7 butterfly stages run in registers as f32x2 operations, 2 as
// shuffles, and no shared memory is passed through.  Reading up to 128 elements a row
// does without the shuffles (see there).
//
// Measured (32 heads x 128, bf16): writing 2048 tokens 17.9 us, 2.4 TB/s, where 6.3 us
// is the moving alone: instructions and the shuffles' rate (one warp's per cycle and SM);
// reading 8192 tokens 42 us, 4.0 TB/s, of which 134 of 170 MB are written.  Single
// tokens of 16 sequences: 4.4 and 5.2 us, latencies.
#include "rq.h"
#include "rq_internal.h"
#include "paged_device.cuh"

namespace rq {
namespace {

constexpr int kPThreads = 128;
constexpr int kMaxTok = 16;          // tokens per block

struct AppendParams {
    const void *x[2];                // K, V
    int64_t token_stride[2], head_stride[2];
    uint8_t *codes[2];
    float *scales[2];
    const int64_t *slots, *positions;
    const uint64_t *turns;
    int64_t tokens, slots_total;     // pages * page_size
    int heads, log_page, half, tb;
    uint64_t seed;
    uint32_t flags;
    float mscale;
};

// How the keys of a block turn: not at all, pairs i and i + half with the whole head
// rotary (a lane then holds both of a pair), with any even part of it, neighbours.
enum Turn { TURN_NONE, TURN_WHOLE, TURN_HALF, TURN_PAIRS };

// The rotary turn of this lane's chunk `ch` (elements 8 ch ..) of a key row.  TURN_HALF
// reads the partner chunk, which a neighbouring lane has just read; half is a multiple of 8.
template <int IN, bool PAIRS>
__device__ __forceinline__ void turn_chunk(const char *row, int ch, const float2 *c, int half, pair_t *v) {
    constexpr int ES = IN == IN_F32 ? 4 : 2;
    const int e0 = 8 * ch;
    if (e0 >= 2 * half) return;
    if constexpr (PAIRS) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 w = c[4 * ch + k];
            const float a = lo2(v[k]), b = hi2(v[k]);
            v[k] = mk2(a * w.x - b * w.y, a * w.y + b * w.x);
        }
    } else {
        const bool first = e0 < half;
        const float sg = first ? -1.f : 1.f;
        pair_t o[4];
        load8<IN>(row + (first ? e0 + half : e0 - half) * ES, o);
        const float4 *cp = reinterpret_cast<const float4 *>(c + (first ? e0 : e0 - half));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 w = cp[k];                       // cos, sin of the pair's two elements
            v[k] = mk2(lo2(v[k]) * w.x + sg * (lo2(o[k]) * w.y), hi2(v[k]) * w.z + sg * (hi2(o[k]) * w.w));
        }
    }
}
// The turn of a whole row whose lanes hold both chunks of each pair: NCH / 2 apart.
template <int D>
__device__ __forceinline__ void turn_row(pair_t (&v)[RowLanes<D>::NP], int rl, const float2 *c) {
    using L = RowLanes<D>;
#pragma unroll
    for (int i = 0; i < L::NCH / 2; ++i) {
        const float4 *cp = reinterpret_cast<const float4 *>(c + 8 * (rl + L::LPR * i));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 w = cp[k];
            const pair_t a = v[4 * i + k], b = v[4 * (i + L::NCH / 2) + k];
            v[4 * i + k] = mk2(lo2(a) * w.x - lo2(b) * w.y, hi2(a) * w.z - hi2(b) * w.w);
            v[4 * (i + L::NCH / 2) + k] = mk2(lo2(b) * w.x + lo2(a) * w.y, hi2(b) * w.z + hi2(a) * w.w);
        }
    }
}

template <int IN, int D, int TURN>
__global__ void __launch_bounds__(kPThreads) kv_append_kernel(const __grid_constant__ AppendParams p) {
    using L = RowLanes<D>;
    constexpr int ES = IN == IN_F32 ? 4 : 2;
    constexpr int RPP = kPThreads / L::LPR;              // rows at a time
    extern __shared__ __align__(16) float2 cs[];         // [tb][half] where keys turn
    __shared__ uint32_t sign_words[8];
    __shared__ int64_t slot_of[kMaxTok];
    const int64_t tok0 = (int64_t)blockIdx.x * p.tb;
    const int nt = (int)min((int64_t)p.tb, p.tokens - tok0);
    const int rl = threadIdx.x % L::LPR, r0 = threadIdx.x / L::LPR;
    const int rows = nt * 2 * p.heads;
    // Row r of the block: token, K or V, head.  A pass's rows are on their way while the
    // pass before it is worked on, the first while the angles are computed.
    struct Row {
        const char *x;
        int tk, h;
        bool is_v;
    };
    auto row_at = [&](int r) {
        Row w;
        w.tk = r / (2 * p.heads);
        const int rest = r - w.tk * 2 * p.heads;
        w.is_v = rest >= p.heads;
        w.h = w.is_v ? rest - p.heads : rest;
        w.x = static_cast<const char *>(p.x[w.is_v]) + ((tok0 + w.tk) * p.token_stride[w.is_v] + w.h * p.head_stride[w.is_v]) * ES;
        return w;
    };
    uint4 raw[L::NCH][ES / 2];
    auto fetch = [&](int r) {
        const char *x = row_at(r).x + rl * 8 * ES;
#pragma unroll
        for (int i = 0; i < L::NCH; ++i)
#pragma unroll
            for (int k = 0; k < ES / 2; ++k)
                raw[i][k] = r < rows ? reinterpret_cast<const uint4 *>(x + L::LPR * i * 8 * ES)[k] : make_uint4(0u, 0u, 0u, 0u);
    };
    fetch(r0);
    block_sign_words<D>(sign_words, p.seed);
    if (threadIdx.x < nt) slot_of[threadIdx.x] = p.slots[tok0 + threadIdx.x];
    if constexpr (TURN != TURN_NONE) {
        for (int i = threadIdx.x; i < nt * p.half; i += kPThreads) {
            const int tk = i / p.half, pr = i - tk * p.half;
            cs[i] = rotary_cos_sin(p.positions[tok0 + tk], p.turns[pr], p.mscale);
        }
    }
    __syncthreads();
    pair_t sg[L::NP];
    row_sign_pairs<D>(sg, sign_words, rl);
    const bool signs_first = (p.flags & RQ_SIGNS_FIRST) != 0;
    constexpr float isd = inv_sqrt_dim<D>();

    // the shuffles name whole warps: every lane runs every pass, rows past the end idle
    for (int base = 0; base < rows; base += RPP) {
        const int r = base + r0;
        const Row w = row_at(r);
        const int64_t slot = r < rows ? slot_of[w.tk] : -1;
        const bool live = slot >= 0 && slot < p.slots_total;   // others are padding
        const bool is_v = w.is_v;
        const int h = w.h;
        pair_t v[L::NP];
#pragma unroll
        for (int i = 0; i < L::NCH; ++i) unpack8<IN>(raw[i], &v[4 * i]);
        fetch(r + RPP);
        if (TURN != TURN_NONE && live && !is_v) {
            const float2 *c = cs + w.tk * p.half;
            if constexpr (TURN == TURN_WHOLE) {
                turn_row<D>(v, rl, c);
            } else {
#pragma unroll
                for (int i = 0; i < L::NCH; ++i) turn_chunk<IN, TURN == TURN_PAIRS>(w.x, rl + L::LPR * i, c, p.half, &v[4 * i]);
            }
        }
        if (signs_first) {
#pragma unroll
            for (int i = 0; i < L::NP; ++i) v[i] ^= sg[i];
        }
        row_fwht<D>(v, rl);
        if (!signs_first) {
#pragma unroll
            for (int i = 0; i < L::NP; ++i) v[i] ^= sg[i];
        }
        float top = pairs_absmax(v);
#pragma unroll
        for (int m = 1; m < L::LPR; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        // A row that holds a NaN or an infinity rotates to nothing but those: its
        // scale becomes NaN, so that it reads back as NaN.
        const float probe = lo2(v[0]);
        const bool bad = !(top < INFINITY) || probe != probe;
        const float inv = top > 0.f && !bad ? fminf(7.0f / top, 3.4028234e38f) : 0.f;
        const pair_t inv2 = mk2(inv, inv), magic = mk2(12582912.f, 12582912.f);   // 1.5 2^23: rounds to nearest even
        if (!live) continue;
        const int64_t at = (((slot >> p.log_page) * p.heads + h) << p.log_page) + (slot & ((1ll << p.log_page) - 1));
        uint32_t *codes = reinterpret_cast<uint32_t *>(p.codes[is_v] + at * (D / 2));
#pragma unroll
        for (int i = 0; i < L::NCH; ++i) {
            uint32_t c[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const pair_t q = fma2(bad ? 0ull : v[4 * i + k], inv2, magic);
                c[2 * k] = (uint32_t)q;
                c[2 * k + 1] = (uint32_t)(q >> 32);
            }
            codes[rl + L::LPR * i] = pack8(c);
        }
        if (rl == 0) p.scales[is_v][at] = bad ? __int_as_float(0x7fffffff) : (top / 7.0f) * isd;
    }
}

struct ReadParams {
    const uint8_t *codes[2];
    const float *scales[2];
    void *out[2];
    const int32_t *table, *starts, *offsets;
    int64_t total, pages, width;
    int heads, log_page, seqs, tb, log_tb;
    uint64_t seed;
    uint32_t flags;
};

// Cache rows of a block's output rows: the row of head 0; -1: no such page (reads
// zeros); -2: not asked for.
__device__ __forceinline__ void read_rows(const ReadParams &p, int64_t n0, int nt, int64_t *at_of) {
    if (threadIdx.x < nt) {
        const int64_t n = n0 + threadIdx.x;
        int lo = 0, hi = p.seqs;             // the last sequence whose first row is at or before n
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.offsets[mid] <= n) lo = mid;
            else hi = mid;
        }
        int64_t at = -2;
        if (n >= p.offsets[lo] && n < p.offsets[lo + 1]) {
            const int64_t pos = n - p.offsets[lo] + (p.starts ? p.starts[lo] : 0);
            const int64_t blk = pos >> p.log_page;
            at = -1;
            if (pos >= 0 && blk < p.width) {
                const int64_t page = p.table[lo * p.width + blk];
                if (page >= 0 && page < p.pages)
                    at = ((page * p.heads) << p.log_page) + (pos & ((1ll << p.log_page) - 1));
            }
        }
        at_of[threadIdx.x] = at;
    }
}

// Rows of up to 128 elements, 16 to a warp, on mma.sync: the codes are exact in fp16 and
// so are the sums of 16 of them in fp32, so a 16-point butterfly is a product with a
// constant +-1 matrix.  A lane (g, c) of rows g and g + 8 holds the code words c, c + 4,
// ... (8 codes each); index bits 0, 2 (the nibbles of a pair are 4 apart) and 3, 4 (c) are
// inside the product, bit 1 and the bits above 4 are left to additions in registers,
// where the results lie.  21 instructions a row; butterflies with shuffles take 41.
template <int OUT, int D>
__global__ void __launch_bounds__(kPThreads) kv_read_mma_kernel(const __grid_constant__ ReadParams p) {
    constexpr int ES = OUT == IN_F32 ? 4 : 2, W = D / 32;            // code words per lane and row
    __shared__ int64_t at_of[kMaxTok];
    __shared__ uint32_t sign_words[4];
    const int64_t n0 = (int64_t)blockIdx.x * p.tb;
    const int nt = (int)min((int64_t)p.tb, p.total - n0);
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    block_sign_words<D>(sign_words, p.seed);
    read_rows(p, n0, nt, at_of);
    __syncthreads();
    const bool rotated = (p.flags & RQ_KV_ROTATED_OUT) != 0;
    const bool signs_first = (p.flags & RQ_SIGNS_FIRST) != 0;        // of R: R^T has them last
    // sign bits of this lane's elements, a byte per word
    uint32_t sgn = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) sgn |= ((sign_words[i] >> (8 * c)) & 0xffu) << (8 * i);
    // B: column n = 8 j + 2 c + i is element bits (0: j, 2: i, 3 4: c); row k = 2 c + i + 8 j alike.
    // This lane: column g of tile j, rows 2 c + {0, 1} and 8 more.
    uint32_t bm[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int kj = 0; kj < 2; ++kj) {
            const uint32_t base = __popc((g >> 1) & c) + (j & kj);
            bm[j][kj] = (base & 1 ? 0xbc00u : 0x3c00u) | ((base + (g & 1)) & 1 ? 0xbc000000u : 0x3c000000u);
        }
    // rows in the order (head, K or V, token): neighbours in a page; tb is a power of two
    const int rows = (2 * p.heads) << p.log_tb;
    constexpr int RPB = 16 * (kPThreads / 32);
    uint32_t cw[2][W];
    float sc[2];
    int64_t at0[2];
    auto fetch = [&](int base) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = base + (threadIdx.x >> 5) * 16 + g + 8 * u;
            const int hs = r >> p.log_tb, tk = r & ((1 << p.log_tb) - 1);
            at0[u] = r < rows && tk < nt ? at_of[tk] : -2;
            sc[u] = 0.f;
#pragma unroll
            for (int i = 0; i < W; ++i) cw[u][i] = 0;
            if (at0[u] >= 0) {
                const int64_t at = at0[u] + ((int64_t)(hs >> 1) << p.log_page);
                sc[u] = p.scales[hs & 1][at];
                const uint32_t *codes = reinterpret_cast<const uint32_t *>(p.codes[hs & 1] + at * (D / 2));
#pragma unroll
                for (int i = 0; i < W; ++i) cw[u][i] = codes[c + 4 * i];
            }
        }
    };
    fetch(0);
    for (int base = 0; base < rows; base += RPB) {
        float v[2 * W][2][4];                // [word, bit 1][bit 0][rows g: bit 2 = 0, 1; rows g + 8]
        float scale[2] = {sc[0], sc[1]};
        int64_t asked[2] = {at0[0], at0[1]};
#pragma unroll
        for (int i = 0; i < W; ++i) {
            uint32_t a[2][4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                code_pairs(cw[u][i], a[u]);  // pairs (e, e + 4), e = 0 .. 3
                if (!rotated && !signs_first) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t b = sgn >> (8 * i + e);
                        a[u][e] ^= ((b & 1u) << 15) | ((b & 16u) << 27);
                    }
                }
            }
#pragma unroll
            for (int b1 = 0; b1 < 2; ++b1) {
                if (rotated) {               // no butterflies: the codes as they are
#pragma unroll
                    for (int j = 0; j < 2; ++j)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&a[u][2 * b1 + j]));
                            v[2 * i + b1][j][2 * u] = f.x;
                            v[2 * i + b1][j][2 * u + 1] = f.y;
                        }
                    continue;
                }
                // k = 2 c + i: bit 2 = i, bit 0 = 0; k + 8: bit 0 = 1
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                                 : "=f"(v[2 * i + b1][j][0]), "=f"(v[2 * i + b1][j][1]), "=f"(v[2 * i + b1][j][2]), "=f"(v[2 * i + b1][j][3])
                                 : "r"(a[0][2 * b1]), "r"(a[1][2 * b1]), "r"(a[0][2 * b1 + 1]), "r"(a[1][2 * b1 + 1]),
                                   "r"(bm[j][0]), "r"(bm[j][1]), "f"(0.f));
            }
        }
        if (base + RPB < rows) fetch(base + RPB);
        if (!rotated) {
#pragma unroll
            for (int st = 1; st < 2 * W; st <<= 1)
#pragma unroll
                for (int i = 0; i < 2 * W; ++i)
                    if (!(i & st)) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int k = 0; k < 4; k += 2) {
                                const float2 x = make_float2(v[i][j][k], v[i][j][k + 1]), y = make_float2(v[i + st][j][k], v[i + st][j][k + 1]);
                                const float2 s = __fadd2_rn(x, y), d = __ffma2_rn(y, make_float2(-1.f, -1.f), x);
                                v[i][j][k] = s.x; v[i][j][k + 1] = s.y;
                                v[i + st][j][k] = d.x; v[i + st][j][k + 1] = d.y;
                            }
                    }
            scale[0] *= inv_sqrt_dim<D>();
            scale[1] *= inv_sqrt_dim<D>();
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (asked[u] < -1) continue;
            const int r = base + (threadIdx.x >> 5) * 16 + g + 8 * u;
            const int hs = r >> p.log_tb, tk = r & ((1 << p.log_tb) - 1);
            char *out = static_cast<char *>(p.out[hs & 1]) + ((n0 + tk) * p.heads + (hs >> 1)) * D * ES;
#pragma unroll
            for (int i = 0; i < W; ++i) {
                pair_t x[4];                 // elements 2 q, 2 q + 1 of the word: bits 2 = q >> 1, 1 = q & 1
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float e0 = v[2 * i + (q & 1)][0][2 * u + (q >> 1)] * scale[u], e1 = v[2 * i + (q & 1)][1][2 * u + (q >> 1)] * scale[u];
                    if (!rotated && signs_first) {
                        const uint32_t b = sgn >> (8 * i + 2 * q);
                        e0 = __uint_as_float(__float_as_uint(e0) ^ (b << 31));
                        e1 = __uint_as_float(__float_as_uint(e1) ^ ((b >> 1) << 31));
                    }
                    x[q] = mk2(e0, e1);
                }
                store8<OUT>(out + (c + 4 * i) * 8 * ES, x);
            }
        }
    }
}

// Rows of 256 elements, by butterflies with shuffles.
template <int OUT, int D>
__global__ void __launch_bounds__(kPThreads) kv_read_kernel(const __grid_constant__ ReadParams p) {
    using L = RowLanes<D>;
    constexpr int ES = OUT == IN_F32 ? 4 : 2;
    constexpr int RPP = kPThreads / L::LPR;
    __shared__ uint32_t sign_words[8];
    __shared__ int64_t at_of[kMaxTok];
    const int64_t n0 = (int64_t)blockIdx.x * p.tb;
    const int nt = (int)min((int64_t)p.tb, p.total - n0);
    block_sign_words<D>(sign_words, p.seed);
    read_rows(p, n0, nt, at_of);
    __syncthreads();
    const int rl = threadIdx.x % L::LPR, r0 = threadIdx.x / L::LPR;
    pair_t sg[L::NP];
    row_sign_pairs<D>(sg, sign_words, rl);
    const bool rotated = (p.flags & RQ_KV_ROTATED_OUT) != 0;
    const bool signs_first = (p.flags & RQ_SIGNS_FIRST) != 0;   // of R: R^T has them last
    constexpr float isd = inv_sqrt_dim<D>();

    // rows in the order (head, K or V, token): consecutive rows lie next to each other in a page
    const int rows = nt * 2 * p.heads;
    for (int base = 0; base < rows; base += RPP) {
        const int r = base + r0;
        const int hs = r / nt, tk = r - hs * nt;
        const int h = hs >> 1, is_v = hs & 1;
        const int64_t at0 = r < rows ? at_of[tk] : -2;
        const int64_t at = at0 + ((int64_t)h << p.log_page);
        pair_t v[L::NP];
        float scale = 0.f;
        if (at0 >= 0) scale = p.scales[is_v][at];
        const uint32_t *codes = reinterpret_cast<const uint32_t *>(p.codes[is_v] + at * (D / 2));
#pragma unroll
        for (int i = 0; i < L::NCH; ++i) {
            const uint32_t w = at0 >= 0 ? codes[rl + L::LPR * i] : 0u;
            pair_t c[4];
            codes_to_pairs(w, c);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[4 * i + k] = c[k];
        }
        if (!rotated) {
            if (!signs_first) {
#pragma unroll
                for (int i = 0; i < L::NP; ++i) v[i] ^= sg[i];
            }
            row_fwht<D>(v, rl);
            if (signs_first) {
#pragma unroll
                for (int i = 0; i < L::NP; ++i) v[i] ^= sg[i];
            }
            scale *= isd;
        }
        if (at0 < -1) continue;
        const pair_t s2 = mk2(scale, scale);
        char *out = static_cast<char *>(p.out[is_v]) + ((n0 + tk) * p.heads + h) * D * ES;
#pragma unroll
        for (int i = 0; i < L::NCH; ++i) {
            pair_t c[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) c[k] = fma2(v[4 * i + k], s2, 0ull);
            store8<OUT>(out + (rl + L::LPR * i) * 8 * ES, c);
        }
    }
}

template <int IN, int D>
cudaError_t launch_append_d(const AppendParams &p, bool rope, bool inter, cudaStream_t stream) {
    const unsigned blocks = (unsigned)((p.tokens + p.tb - 1) / p.tb);
    const size_t smem = rope ? sizeof(float2) * p.tb * p.half : 0;
    if (!rope) {
        kv_append_kernel<IN, D, TURN_NONE><<<blocks, kPThreads, 0, stream>>>(p);
    } else if (inter) {
        kv_append_kernel<IN, D, TURN_PAIRS><<<blocks, kPThreads, smem, stream>>>(p);
    } else {
        if constexpr (D >= 64) {
            if (2 * p.half == D) {
                kv_append_kernel<IN, D, TURN_WHOLE><<<blocks, kPThreads, smem, stream>>>(p);
                return cudaGetLastError();
            }
        }
        kv_append_kernel<IN, D, TURN_HALF><<<blocks, kPThreads, smem, stream>>>(p);
    }
    return cudaGetLastError();
}
template <int IN>
cudaError_t launch_append_in(const AppendParams &p, int64_t d, bool rope, bool inter, cudaStream_t stream) {
    switch (d) {
        case 32: return launch_append_d<IN, 32>(p, rope, inter, stream);
        case 64: return launch_append_d<IN, 64>(p, rope, inter, stream);
        case 128: return launch_append_d<IN, 128>(p, rope, inter, stream);
        default: return launch_append_d<IN, 256>(p, rope, inter, stream);
    }
}
template <int OUT>
cudaError_t launch_read_out(const ReadParams &p, int64_t d, cudaStream_t stream) {
    const unsigned blocks = (unsigned)((p.total + p.tb - 1) / p.tb);
    switch (d) {
        case 32: kv_read_mma_kernel<OUT, 32><<<blocks, kPThreads, 0, stream>>>(p); break;
        case 64: kv_read_mma_kernel<OUT, 64><<<blocks, kPThreads, 0, stream>>>(p); break;
        case 128: kv_read_mma_kernel<OUT, 128><<<blocks, kPThreads, 0, stream>>>(p); break;
        default: kv_read_kernel<OUT, 256><<<blocks, kPThreads, 0, stream>>>(p); break;
    }
    return cudaGetLastError();
}

int log2_of(int64_t n) {
    int l = 0;
    while ((int64_t(1) << l) < n) ++l;
    return l;
}

}  // namespace

cudaError_t launch_kv_append(const KvRows &k, const KvRows &v, int in_type, int64_t tokens, int64_t head_dim,
                             const PagedCache &c, const int64_t *slots, const int64_t *positions,
                             const uint64_t *turns, int64_t rot, float mscale, bool inter, uint64_t seed,
                             uint32_t flags, cudaStream_t stream) {
    AppendParams p{};
    p.x[0] = k.x;
    p.x[1] = v.x;
    p.token_stride[0] = k.token_stride;
    p.token_stride[1] = v.token_stride;
    p.head_stride[0] = k.head_stride;
    p.head_stride[1] = v.head_stride;
    p.codes[0] = c.kq;
    p.codes[1] = c.vq;
    p.scales[0] = c.ks;
    p.scales[1] = c.vs;
    p.slots = slots;
    p.positions = positions;
    p.turns = turns;
    p.tokens = tokens;
    p.slots_total = c.pages * c.page_size;
    p.heads = (int)c.heads;
    p.log_page = log2_of(c.page_size);
    p.half = (int)(rot / 2);
    p.seed = seed;
    p.flags = flags;
    p.mscale = mscale;
    // as many tokens per block as leave every SM eight (cache of 32 heads x 128, 2048 bf16
    // tokens: 17.9 us; with 4 blocks 18.9, with 16 19.8)
    const int64_t want = 8 * (int64_t)device_sm_count();
    p.tb = (int)((tokens + want - 1) / want);
    if (p.tb > kMaxTok) p.tb = kMaxTok;
    if ((tokens + p.tb - 1) / p.tb > 0x7fffffffll) return cudaErrorInvalidValue;
    const bool rope = turns != nullptr;
    switch (in_type) {
        case IN_F32: return launch_append_in<IN_F32>(p, head_dim, rope, inter, stream);
        case IN_BF16: return launch_append_in<IN_BF16>(p, head_dim, rope, inter, stream);
        default: return launch_append_in<IN_F16>(p, head_dim, rope, inter, stream);
    }
}

cudaError_t launch_kv_read(const PagedCache &c, int64_t head_dim, const int32_t *table, int64_t width,
                           const int32_t *starts, const int32_t *offsets, int64_t seqs, int64_t total, uint64_t seed,
                           uint32_t flags, void *k_out, void *v_out, int out_type, cudaStream_t stream) {
    ReadParams p{};
    p.codes[0] = c.kq;
    p.codes[1] = c.vq;
    p.scales[0] = c.ks;
    p.scales[1] = c.vs;
    p.out[0] = k_out;
    p.out[1] = v_out;
    p.table = table;
    p.starts = starts;
    p.offsets = offsets;
    p.total = total;
    p.pages = c.pages;
    p.width = width;
    p.heads = (int)c.heads;
    p.log_page = log2_of(c.page_size);
    p.seqs = (int)seqs;
    p.seed = seed;
    p.flags = flags;
    p.tb = kMaxTok;
    const int64_t want = 8 * (int64_t)device_sm_count();
    while (p.tb > 1 && total / p.tb < want) p.tb /= 2;
    p.log_tb = log2_of(p.tb);
    if ((total + p.tb - 1) / p.tb > 0x7fffffffll) return cudaErrorInvalidValue;
    switch (out_type) {
        case IN_F32: return launch_read_out<IN_F32>(p, head_dim, stream);
        case IN_BF16: return launch_read_out<IN_BF16>(p, head_dim, stream);
        default: return launch_read_out<IN_F16>(p, head_dim, stream);
    }
}

}  // namespace rq
