// rope.cu -- rotary positions on the rows of Q and K (sm_103a).
//
// The first `rot` of a head's D elements are rot/2 pairs (a, b): (i, i + rot/2) in the
// half layout, (2i, 2i + 1) in the interleaved one.  Pair i of a token at position t
// turns by t w_i (the transposed turn with RQ_ROPE_INVERSE, which is the gradient):
//   a' = (a cos - b sin) m,  b' = (a sin + b cos) m;   the other D - rot elements pass.
//
// Bound by reading and writing the rows once.  One block covers a few tokens and all
// heads of Q and K: it computes the tokens' cosines and sines once into shared memory
// (see rotary_cos_sin: no table of positions is read), then its threads stream the
// head rows, each thread always the same 16-byte piece (or pair of pieces) of a row.
// Rows whose addresses or rot do not allow 16-byte pieces go element by element.
//
// Measured: 65,536 tokens of 32 + 8 heads x 128 (bf16) 227 us, 5.9 TB/s, 0.87 of a copy's
// rate; two rows in flight per thread, as one gives 232 us and four 249.  One token: 4 us,
// its latencies; a call's host side takes 17.
#include "rq.h"
#include "rq_internal.h"
#include "paged_device.cuh"

namespace rq {
namespace {

constexpr int kRThreads = 256;

struct RParams {
    RopeView t[2];          // Q, then K (heads 0: absent)
    const int64_t *positions;
    const uint64_t *turns;
    int64_t tokens;
    int head_dim, half;     // half = rot / 2
    int tb;                 // tokens per block
    int items, rot_items;   // pieces of a row, and how many of them rotate
    float mscale, sgn;      // sgn: +1, or -1 for the transposed turn
};

// VEC: pieces of 16 bytes (8 or 4 elements); otherwise one pair or one element each.
template <int IN, bool INTER, bool VEC>
__global__ void __launch_bounds__(kRThreads) rope_kernel(const __grid_constant__ RParams p) {
    constexpr int ES = IN == IN_F32 ? 4 : 2;
    constexpr int VE = VEC ? 16 / ES : (INTER ? 2 : 1);   // elements of a piece
    extern __shared__ float2 cs[];                        // [tb][half]
    const int64_t tok0 = (int64_t)blockIdx.x * p.tb;
    const int nt = (int)min((int64_t)p.tb, p.tokens - tok0);
    for (int i = threadIdx.x; i < nt * p.half; i += kRThreads) {
        const int tk = i / p.half, pr = i - tk * p.half;
        float2 v = rotary_cos_sin(p.positions[tok0 + tk], p.turns[pr], p.mscale);
        v.y *= p.sgn;
        cs[i] = v;
    }
    __syncthreads();
    const int heads = (int)(p.t[0].heads + p.t[1].heads);
    const int rpp = kRThreads / p.items;                  // rows at a time
    const int r0 = threadIdx.x / p.items, it = threadIdx.x - r0 * p.items;
    if (r0 >= rpp) return;
    const bool turn = it < p.rot_items;
    // element offsets of this thread's piece(s) in a row
    const int ea = turn ? it * VE : 2 * p.half + (it - p.rot_items) * VE;
    const int eb = ea + p.half;
    const int rows = nt * heads;
    constexpr int U = VEC ? 2 : 1;                        // rows in flight per thread
    for (int rb = r0; rb < rows; rb += U * rpp) {
        const char *src[U];
        char *dst[U];
        const float2 *c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = rb + u * rpp;
            const int tk = r / heads;
            int h = r - tk * heads;
            const bool second = h >= p.t[0].heads;
            const RopeView &v = p.t[second];
            if (second) h -= (int)p.t[0].heads;
            src[u] = static_cast<const char *>(v.src) + ((tok0 + tk) * v.src_token + h * v.src_head) * ES;
            dst[u] = static_cast<char *>(v.dst) + ((tok0 + tk) * v.dst_token + h * v.dst_head) * ES;
            c[u] = cs + tk * p.half;
        }
        if constexpr (VEC) {
            uint4 ra[U], rc[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (rb + u * rpp < rows) {
                    ra[u] = *reinterpret_cast<const uint4 *>(src[u] + ea * ES);
                    if (!INTER && turn) rc[u] = *reinterpret_cast<const uint4 *>(src[u] + eb * ES);
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (rb + u * rpp >= rows) break;
                if (!turn) {
                    *reinterpret_cast<uint4 *>(dst[u] + ea * ES) = ra[u];
                    continue;
                }
                float a[VE], b[VE], oa[VE], ob[VE];
                unpack16<IN>(ra[u], a);
                if constexpr (!INTER) {
                    unpack16<IN>(rc[u], b);
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float2 w = c[u][ea + e];
                        oa[e] = a[e] * w.x - b[e] * w.y;
                        ob[e] = a[e] * w.y + b[e] * w.x;
                    }
                    *reinterpret_cast<uint4 *>(dst[u] + ea * ES) = pack16<IN>(oa);
                    *reinterpret_cast<uint4 *>(dst[u] + eb * ES) = pack16<IN>(ob);
                } else {
#pragma unroll
                    for (int e = 0; e < VE; e += 2) {
                        const float2 w = c[u][(ea + e) / 2];
                        oa[e] = a[e] * w.x - a[e + 1] * w.y;
                        oa[e + 1] = a[e] * w.y + a[e + 1] * w.x;
                    }
                    *reinterpret_cast<uint4 *>(dst[u] + ea * ES) = pack16<IN>(oa);
                }
            }
        } else if (!turn) {
#pragma unroll
            for (int e = 0; e < VE; ++e) store_elem<IN>(dst[0], ea + e, load_elem<IN>(src[0], ea + e));
        } else {
            const int ia = ea, ib = INTER ? ea + 1 : eb;
            const float a = load_elem<IN>(src[0], ia), b = load_elem<IN>(src[0], ib);
            const float2 w = c[0][it];
            store_elem<IN>(dst[0], ia, a * w.x - b * w.y);
            store_elem<IN>(dst[0], ib, a * w.y + b * w.x);
        }
    }
}

template <int IN>
cudaError_t launch_rope_in(RParams &p, bool inter, bool vec, int rot, cudaStream_t stream) {
    const int ve = vec ? (IN == IN_F32 ? 4 : 8) : (inter ? 2 : 1);
    p.rot_items = (inter ? rot : rot / 2) / ve;
    p.items = p.rot_items + (p.head_dim - rot) / ve;
    // as many tokens per block as there are threads for their pairs, fewer while
    // that leaves SMs without a full set of blocks
    const int64_t want = 8 * (int64_t)device_sm_count();
    p.tb = kRThreads / p.half;
    if (p.tb < 1) p.tb = 1;
    while (p.tb > 1 && p.tokens / p.tb < want) p.tb /= 2;
    const int64_t blocks = (p.tokens + p.tb - 1) / p.tb;
    if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
    const size_t smem = sizeof(float2) * p.tb * p.half;
    const dim3 grid((unsigned)blocks);
    if (vec) {
        if (inter) rope_kernel<IN, true, true><<<grid, kRThreads, smem, stream>>>(p);
        else rope_kernel<IN, false, true><<<grid, kRThreads, smem, stream>>>(p);
    } else {
        if (inter) rope_kernel<IN, true, false><<<grid, kRThreads, smem, stream>>>(p);
        else rope_kernel<IN, false, false><<<grid, kRThreads, smem, stream>>>(p);
    }
    return cudaGetLastError();
}

bool vec16(const RopeView &v, int es) {
    if (!v.heads) return true;
    const uint64_t bits = reinterpret_cast<uint64_t>(v.src) | reinterpret_cast<uint64_t>(v.dst) |
                          (uint64_t)(v.src_token * es) | (uint64_t)(v.src_head * es) | (uint64_t)(v.dst_token * es) |
                          (uint64_t)(v.dst_head * es);
    return (bits & 15) == 0;
}

}  // namespace

cudaError_t launch_rope(const RopeView &q, const RopeView &k, int in_type, int64_t tokens, int64_t head_dim,
                        int64_t rot, const int64_t *positions, const uint64_t *turns, float mscale, bool inter,
                        bool inverse, cudaStream_t stream) {
    RParams p{};
    p.t[0] = q;
    p.t[1] = k;
    p.positions = positions;
    p.turns = turns;
    p.tokens = tokens;
    p.head_dim = (int)head_dim;
    p.half = (int)(rot / 2);
    p.mscale = mscale;
    p.sgn = inverse ? -1.f : 1.f;
    const int es = in_type == IN_F32 ? 4 : 2, ve = 16 / es;
    const bool vec = vec16(q, es) && vec16(k, es) && (inter ? rot : rot / 2) % ve == 0 && (head_dim - rot) % ve == 0;
    switch (in_type) {
        case IN_F32: return launch_rope_in<IN_F32>(p, inter, vec, (int)rot, stream);
        case IN_BF16: return launch_rope_in<IN_BF16>(p, inter, vec, (int)rot, stream);
        default: return launch_rope_in<IN_F16>(p, inter, vec, (int)rot, stream);
    }
}

}  // namespace rq
