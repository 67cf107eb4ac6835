// w4a16_gemm.cu -- products of a few rows of activations with 4-bit weights (sm_103a).
//
//   y[m][c] = sum_g s[c][g] sum_{k in g} x[m][k] q[c][k]      (g: 128 codes, or the channel)
// x is not quantised: its elements enter the tensor cores as fp16, bf16 and fp32 rows relative
// to a power of two for each 128 of them (the largest becomes 2^14 or more).  bf16's 8 bits are
// exact there down to 2^-31 of the largest, fp32 goes in two parts, 22 bits; codes are exact,
// so the products are too.
//
// Bound by reading the weights once, so they stream straight into registers, several items
// ahead.  An item is 16 channels x 128 codes, 32 bytes a lane.  A block per SM owns a run of
// channels and goes over them in turn; its 16 warps split K and, where that leaves them enough
// to do, the channels, and meet in shared memory once per channel.
//  * mma.sync m16n8k16, channels x rows.  A lane's 16 bytes of a channel's step are codes
//    32 c .. 32 c + 31 (c = lane % 4): words of 8 codes whose nibbles j and j + 4 are a pair of
//    operands.  The rows lie in shared memory in that order, 16 bytes to a word, placed so
//    that a warp's reads are free of bank conflicts.
//  * an item's sums of 128 products begin from 0 in the tensor core (whose additions are not
//    rounded to nearest) and are scaled and added in fp32 outside.
//  * rows that do not fit shared memory, or take long to get there, split K over a cluster of
//    CTAs, whose sums meet in distributed shared memory; more than 16 rows take the weights
//    again, from L2 (32 rows at a time spill registers: 61 rows 67 us for 60).
// Measured, groups of 128, weights from HBM (L2 flushed) and in brackets on the same inputs, where those of
// the first two lie in L2: 1 row, 4096 -> 14336, 11.8 us (9.6), 2.6 TB/s of weights and scales; 7 rows,
// 14336 -> 4096, 14.1 us (11.6); 16 rows, 8192 -> 28672, 42.5 us (40.5), 3.0 TB/s.  What it spends them on there:
// issue slots are 48% busy, 201 instructions for a warp's step of 16 x 128 codes (some 90 to widen
// them, 16 products, 8 reads of the rows), and 16 warps, all that fit, do not hide the rest.
// Without the weights' loads it takes 36 us, without products and widening 37, without
// either 22.  Equal stretches of all steps for each warp, which meet at the end only, were no
// faster (43.4 us; 1 row 11.9).
#include "rq.h"
#include "rq_internal.h"
#include "paged_device.cuh"

namespace rq {
namespace {

constexpr int kGWarps = 16, kGThreads = 32 * kGWarps;
constexpr int kItem = 4;                // steps of a warp's item: what it computes, and has in flight
constexpr int kSumBlocks = 16;          // blocks of 16 channels and one other warp whose sums wait for the cluster

constexpr int kMostBytes = 227 * 1024;

struct W16Params {
    const void *x;
    const uint8_t *w;
    const float *s;
    void *y;
    int64_t M, N, K, ldx;
    int out;                    // InType of y
    bool grouped;
    int steps;                  // 128-code steps of K
    int rows;                   // of a block
    int log_ks;                 // log2 of the CTAs of a cluster
    int log_kw, per;            // log2 of the warps that split K; a warp's steps of each kw * per
    int blocks;                 // of 16 channels for each of the other warps
    int each, more;             // blocks of a cluster; the first `more` have one more
    int64_t block_bytes, block_scales;      // from a block's lines of weights, and scales, to the next's
    bool scales4;               // an item's scales are 16 bytes at a 16-byte boundary
    uint32_t row_bytes;         // of a row in shared memory, 64 more than a multiple of 128
};

template <bool FIRST>
__device__ __forceinline__ void mma_w16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (FIRST)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 elements of a row as they lie in memory.
template <int IN>
struct RowChunk {
    uint4 v[IN == IN_F32 ? 2 : 1];
};
template <int IN>
__device__ __forceinline__ RowChunk<IN> row_chunk(const void *row, int64_t at) {
    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(row) + at * (IN == IN_F32 ? 4 : 2));
    RowChunk<IN> c;
#pragma unroll
    for (int i = 0; i < (IN == IN_F32 ? 2 : 1); ++i) c.v[i] = p[i];
    return c;
}

// The same as fp16 in the order of a word's pairs, part h of (element j, element j + 4); bf16 and
// fp32 times 1 / *unit, a power of two that the 16 threads of a step agree on (`mask`: their lanes).
template <int IN, int PARTS>
__device__ __forceinline__ float row_pairs(const RowChunk<IN> &r, uint32_t mask, uint4 (&b)[PARTS]) {
    if constexpr (IN == IN_F16) {
        const uint4 v = r.v[0];
        b[0] = make_uint4(__byte_perm(v.x, v.z, 0x5410u), __byte_perm(v.x, v.z, 0x7632u), __byte_perm(v.y, v.w, 0x5410u),
                          __byte_perm(v.y, v.w, 0x7632u));
        return 1.f;
    } else {
        float x[8];
        uint32_t top = 0;
        if constexpr (IN == IN_F32) {
            const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[j] = __uint_as_float(w[j]);
                top = max(top, w[j] & 0x7fffffffu);
            }
        } else {
            unpack16<IN_BF16>(r.v[0], x);
            auto size = [](uint32_t w) { return __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w)); };
            const __nv_bfloat162 m = __hmax2(__hmax2(size(r.v[0].x), size(r.v[0].y)), __hmax2(size(r.v[0].z), size(r.v[0].w)));
            const uint32_t both = *reinterpret_cast<const uint32_t *>(&m);
            top = max(both << 16, both & 0xffff0000u);
        }
        top = __reduce_max_sync(mask, top);
        // 2^ex > the largest; at least what leaves 2^(15 - ex) a float
        const int ex = max(-111, (int)(top >> 23) - 126);
        const float down = __uint_as_float((uint32_t)(127 + 15 - ex) << 23), up = __uint_as_float((uint32_t)(127 - 15 + ex) << 23);
        uint32_t h[PARTS][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo = x[j] * down, hi = x[j + 4] * down;
#pragma unroll
            for (int i = 0; i < PARTS; ++i) {
                const __half2 v = __floats2half2_rn(lo, hi);
                h[i][j] = *reinterpret_cast<const uint32_t *>(&v);
                const float2 got = __half22float2(v);
                lo -= got.x;
                hi -= got.y;
            }
        }
#pragma unroll
        for (int i = 0; i < PARTS; ++i) b[i] = make_uint4(h[i][0], h[i][1], h[i][2], h[i][3]);
        return up;
    }
}

__device__ __forceinline__ uint4 ld_weights(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A float of CTA `rank` of the cluster, where this one has `local`.
__device__ __forceinline__ float cluster_load(const float *local, int rank) {
    uint32_t remote;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"((uint32_t)__cvta_generic_to_shared(local)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(remote) : "memory");
    return v;
}

template <int IN, int MT>
__global__ void __launch_bounds__(kGThreads, 1) w4a16_kernel(const __grid_constant__ W16Params p) {
    constexpr int PARTS = IN == IN_F32 ? 2 : 1, ES = IN == IN_F32 ? 4 : 2, RM = 8 * MT;
    constexpr bool UNIT = IN != IN_F16;
    extern __shared__ uint8_t raw[];
    // the warps' sums, twice [warp][row][channel]; the cluster's; the rows; their units
    float(*part)[kGWarps][16 * RM] = reinterpret_cast<float(*)[kGWarps][16 * RM]>(raw);
    float *const sums = reinterpret_cast<float *>(raw + sizeof(float) * 2 * kGWarps * 16 * RM);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    const int kw = 1 << p.log_kw, log_cw = 4 - p.log_kw, cw = 1 << log_cw, wk = warp & (kw - 1), wc = warp >> p.log_kw;
    const int ks = 1 << p.log_ks, rank = blockIdx.x & (ks - 1), cluster = blockIdx.x >> p.log_ks;
    uint8_t *const rows = reinterpret_cast<uint8_t *>(sums + (ks > 1 ? kSumBlocks * 16 * RM : 0));
    const int m0 = blockIdx.y * p.rows, M = min(p.rows, (int)p.M - m0);
    float *const units = reinterpret_cast<float *>(rows + PARTS * M * p.row_bytes);       // [step][row]
    const int blk0 = p.each * cluster + min(cluster, p.more), nb = p.each + (cluster < p.more);
    const uint32_t N = (uint32_t)p.N;
    const int stride = p.per << p.log_kw;                        // steps of an item of all warps
    const int s0 = (int)((int64_t)p.steps * rank >> p.log_ks), ns = (int)((int64_t)p.steps * (rank + 1) >> p.log_ks) - s0;

    // the item on its way: its weights, a step's as soon as the one before it has left their place, and its
    // scales; steps at .. at + n - 1 of the CTA's, of the block whose lines begin at w0
    uint4 a[kItem][2];
    float f[kItem][2];
    const int at0 = wk * p.per;
    int at = at0, n, loads = nb;                         // blocks whose items are still to be loaded
    uint32_t pn = (uint32_t)(blk0 * cw + wc) * 16 + g;
    const uint8_t *w0;
    const float *f0;
    uint32_t w8, f8;                                     // from there to the line 8 channels on
    auto channels = [&] {                                // past N: the last, never stored
        const uint32_t ch0 = min(pn, N - 1), next = min(pn + 8, N - 1) - ch0;
        w0 = p.w + (int64_t)ch0 * (p.K / 2) + (s0 + at0) * 64 + 16 * c;
        w8 = next * (uint32_t)(p.K / 2);
        f0 = p.grouped ? p.s + (int64_t)ch0 * p.steps + s0 + at0 : p.s + ch0;
        f8 = next * (p.grouped ? p.steps : 1);
    };
    auto weights = [&](int j) {
        if (j < n) {
            a[j][0] = ld_weights(w0 + 64 * j);
            a[j][1] = ld_weights(w0 + w8 + 64 * j);
        }
    };
    auto scales = [&] {
        if (p.scales4 && n == kItem) {
            const float4 x = *reinterpret_cast<const float4 *>(f0), y = *reinterpret_cast<const float4 *>(f0 + f8);
            f[0][0] = x.x; f[1][0] = x.y; f[2][0] = x.z; f[3][0] = x.w;
            f[0][1] = y.x; f[1][1] = y.y; f[2][1] = y.z; f[3][1] = y.w;
        } else {
#pragma unroll
            for (int j = 0; j < kItem; ++j)
                if (j < n) {
                    f[j][0] = f0[p.grouped ? j : 0];
                    f[j][1] = (f0 + f8)[p.grouped ? j : 0];
                }
        }
    };
    auto next = [&] {                                    // to the item after this one
        at += stride;
        if (at - at0 < ns) {
            w0 += stride * 64;
            f0 += p.grouped ? stride : 0;
        } else {                                         // of the next block
            w0 += p.block_bytes - (at - stride - at0) * 64;
            f0 += p.block_scales - (p.grouped ? at - stride - at0 : 0);
            at = at0;
            --loads;
            pn += 16 * cw;
            if (pn + 8 >= N) channels();
        }
        n = loads > 0 ? min(p.per, ns - at) : 0;
    };
    channels();
    n = min(p.per, ns - at);
#pragma unroll
    for (int j = 0; j < kItem; ++j) weights(j);
    scales();
    // the rows, word by word, while the first items are on their way; 16 threads to a step
    constexpr int U = IN == IN_F32 ? 4 : 8;
    for (int ch = threadIdx.x; ch - lane < ns * 16; ch += kGThreads) {       // whole warps
        const int at = (ch & ~15) + ((ch & 3) << 2) + ((ch >> 2) & 3);       // step, word, lane column
        const bool there = ch < ns * 16;
        const char *src = static_cast<const char *>(p.x) + ((int64_t)m0 * p.ldx + (int64_t)s0 * 128 + 8 * (there ? ch : 0)) * ES;
        for (int mm = 0; mm < M; mm += U) {
            RowChunk<IN> r[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (mm + u < M) r[u] = row_chunk<IN>(src + (mm + u) * p.ldx * ES, 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (mm + u >= M) break;
                uint4 b[PARTS];
                const float up = row_pairs<IN, PARTS>(r[u], lane < 16 ? 0x0000ffffu : 0xffff0000u, b);
                if (!there) continue;
#pragma unroll
                for (int h = 0; h < PARTS; ++h)
                    *reinterpret_cast<uint4 *>(rows + (h * M + mm + u) * p.row_bytes + at * 16) = b[h];
                if (UNIT && (ch & 15) == 0) units[(ch >> 4) * RM + mm + u] = up;
            }
        }
    }
    __syncthreads();

    // a lane's row of each n8 tile; what stands for rows that are not there reaches no row that is
    const uint8_t *row[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) row[t] = rows + min(8 * t + g, M - 1) * p.row_bytes + 16 * c;
    float sum[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int k = 0; k < 4; ++k) sum[t][k] = 0.f;
#pragma unroll 1
    for (int b = 0; b < nb; ++b) {
#pragma unroll 1
        for (int i0 = 0; i0 < ns; i0 += stride) {
            float xf[kItem][2];
#pragma unroll
            for (int j = 0; j < kItem; ++j)
#pragma unroll
                for (int k = 0; k < 2; ++k) xf[j][k] = f[j][k];
            const int i1 = i0 + at0, here = n;
            next();
            scales();
#pragma unroll
            for (int j = 0; j < kItem; ++j) {
                if (j >= here) {
                    weights(j);
                    continue;
                }
                const uint32_t x0[4] = {a[j][0].x, a[j][0].y, a[j][0].z, a[j][0].w}, x1[4] = {a[j][1].x, a[j][1].y, a[j][1].z, a[j][1].w};
                float o[MT][4];
#pragma unroll
                for (int wd = 0; wd < 4; ++wd) {
                    uint32_t q0[4], q1[4];
                    code_pairs(x0[wd], q0);
                    code_pairs(x1[wd], q1);
                    const uint32_t a0[4] = {q0[0], q1[0], q0[1], q1[1]}, a1[4] = {q0[2], q1[2], q0[3], q1[3]};
#pragma unroll
                    for (int h = PARTS - 1; h >= 0; --h)                 // the small part first
#pragma unroll
                        for (int t = 0; t < MT; ++t) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(
                                row[t] + (uint32_t)i1 * 256u + (uint32_t)(h * M) * p.row_bytes + (j * 256 + wd * 64));
                            if (wd == 0 && h == PARTS - 1) mma_w16<true>(o[t], a0, v.x, v.y);
                            else mma_w16<false>(o[t], a0, v.x, v.y);
                            mma_w16<false>(o[t], a1, v.z, v.w);
                        }
                }
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    // the weights' scale first: a unit alone may leave fp32's range
                    float2 e = make_float2(1.f, 1.f);
                    if constexpr (UNIT) e = *reinterpret_cast<const float2 *>(units + (i1 + j) * RM + 8 * t + 2 * c);
                    sum[t][0] = fmaf(o[t][0] * xf[j][0], e.x, sum[t][0]);
                    sum[t][1] = fmaf(o[t][1] * xf[j][0], e.y, sum[t][1]);
                    sum[t][2] = fmaf(o[t][2] * xf[j][1], e.x, sum[t][2]);
                    sum[t][3] = fmaf(o[t][3] * xf[j][1], e.y, sum[t][3]);
                }
                weights(j);
            }
        }
        // the block's sums, from its warps
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (8 * t + 2 * c + (k & 1) < M) part[b & 1][warp][(8 * t + 2 * c + (k & 1)) * 16 + g + 8 * (k >> 1)] = sum[t][k];
                sum[t][k] = 0.f;
            }
        __syncthreads();
        auto store = [&](int e, int64_t block, float v) {                // element (row, other warp, channel) of a block
            const int64_t ch = (block << (log_cw + 4)) + (e & ((16 << log_cw) - 1));
            if (ch >= p.N) return;
            const int64_t out = (m0 + (e >> (log_cw + 4))) * p.N + ch;
            if (p.out == IN_F32) store_elem<IN_F32>(p.y, out, v);
            else if (p.out == IN_BF16) store_elem<IN_BF16>(p.y, out, v);
            else store_elem<IN_F16>(p.y, out, v);
        };
        const int wait = ks > 1 ? kSumBlocks >> log_cw : 1, slot = b % wait, each = M << (log_cw + 4);
        for (int e = threadIdx.x; e < each; e += kGThreads) {
            const float *src = &part[b & 1][((e >> 4) & (cw - 1)) << p.log_kw][(e >> (log_cw + 4)) * 16 + (e & 15)];
            float v = 0.f;
            for (int w = 0; w < kw; ++w) v += src[w * 16 * RM];
            if (ks > 1) sums[slot * each + e] = v;
            else store(e, blk0 + b, v);
        }
        if (ks > 1 && (slot == wait - 1 || b == nb - 1)) {               // each CTA adds up its share of the cluster's
            cluster_sync();
            for (int e = rank * kGThreads + threadIdx.x; e < (slot + 1) * each; e += ks * kGThreads) {
                float v = 0.f;
                for (int r = 0; r < ks; ++r) v += cluster_load(sums + e, r);
                const int bb = e / each;
                store(e - bb * each, blk0 + b - slot + bb, v);
            }
            cluster_sync();
        }
    }
}

// The current device.
struct W16Device {
    int id, sms;
};

// Clusters of 2^log_ks such CTAs that it holds at once; 0 on error.
template <int IN, int MT>
int w16_clusters(const W16Device &dev, int log_ks) {
    static std::atomic<int> known[kMaxDevices][4];
    if (log_ks == 0) return dev.sms;
    int n = 0;
    if (dev.id < kMaxDevices && (n = known[dev.id][log_ks].load(std::memory_order_relaxed))) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(dev.sms >> log_ks << log_ks);
    cfg.blockDim = dim3(kGThreads);
    cfg.dynamicSmemBytes = kMostBytes;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {1u << log_ks, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, w4a16_kernel<IN, MT>, &cfg) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        return 0;
    }
    if (dev.id < kMaxDevices) known[dev.id][log_ks].store(n, std::memory_order_relaxed);
    return n;
}

// How a call is split: the one with the least to do for the fullest CTA, in steps of its 16
// warps (about 0.35 us): half a step for an item's own cost and one for a block's, the rows'
// way into shared memory (16 KB a step), four steps for a cluster's meeting.  false: the
// rows fit no cluster's shared memory.
template <int IN, int MT>
bool w16_split(const W16Device &dev, W16Params &p, size_t &bytes) {
    constexpr int RM = 8 * MT, PARTS = IN == IN_F32 ? 2 : 1;
    double least = 1e30;
    for (int log_ks = 0; log_ks <= 3 && (1 << log_ks) <= p.steps; ++log_ks) {
        const int clusters = w16_clusters<IN, MT>(dev, log_ks), steps = (p.steps + (1 << log_ks) - 1) >> log_ks;
        const int64_t row_bytes = (int64_t)steps * 256 + 64, rows = PARTS * p.rows * row_bytes;
        const int64_t need = (int64_t)sizeof(float) * (2 * kGWarps + (log_ks ? kSumBlocks : 0)) * 16 * RM + rows + (int64_t)steps * RM * sizeof(float);
        if (clusters <= 0 || need > kMostBytes) continue;
        for (int log_kw = 4; log_kw >= 0; --log_kw) {
            const int64_t cw = kGWarps >> log_kw, blocks = (p.N + 16 * cw - 1) / (16 * cw);
            const int each = (steps + (1 << log_kw) - 1) >> log_kw, per = each < kItem ? each : kItem;
            const double cost = (double)((blocks + clusters - 1) / clusters) * ((each + per - 1) / per * (per + 0.5) + 1.0) +
                                (double)rows / 16384 + (log_ks ? 4.0 : 0.0);
            if (cost >= least) continue;
            least = cost;
            p.log_ks = log_ks;
            p.log_kw = log_kw;
            p.per = per;
            p.blocks = (int)blocks;
            p.row_bytes = (uint32_t)row_bytes;
            bytes = (size_t)need;
        }
    }
    return least < 1e30;
}

template <int IN, int MT>
cudaError_t launch_w16_m(const W16Device &dev, W16Params p, cudaStream_t stream) {
    auto kern = w4a16_kernel<IN, MT>;
    static std::atomic<uint64_t> allowed;
    cudaError_t e = allow_smem((const void *)kern, kMostBytes, allowed);
    if (e != cudaSuccess) return e;
    p.steps = (int)(p.K / 128);
    size_t bytes = 0;
    p.rows = (int)(p.M < 8 * MT ? p.M : 8 * MT);
    while (!w16_split<IN, MT>(dev, p, bytes)) {                                       // fewer rows at a time
        if constexpr (MT > 1) return launch_w16_m<IN, MT / 2>(dev, p, stream);
        if (p.rows == 1) return cudaErrorInvalidValue;
        p.rows /= 2;
    }
    const int cw = kGWarps >> p.log_kw, most = w16_clusters<IN, MT>(dev, p.log_ks), clusters = p.blocks < most ? p.blocks : most;
    p.block_bytes = p.K / 2 * 16 * cw;
    p.block_scales = (p.grouped ? p.steps : 1) * 16 * cw;
    p.scales4 = p.grouped && p.per == kItem && p.steps % (kItem << p.log_ks) == 0 && reinterpret_cast<uintptr_t>(p.s) % 16 == 0;
    p.each = p.blocks / clusters;
    p.more = p.blocks % clusters;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(clusters << p.log_ks), (unsigned)((p.M + p.rows - 1) / p.rows));
    cfg.blockDim = dim3(kGThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {1u << p.log_ks, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int IN>
cudaError_t launch_w16(const W16Params &p, cudaStream_t stream) {
    W16Device dev{0, device_sm_count()};
    if (dev.sms <= 0 || cudaGetDevice(&dev.id) != cudaSuccess) return cudaErrorUnknown;
    return p.M <= 8 ? launch_w16_m<IN, 1>(dev, p, stream) : launch_w16_m<IN, 2>(dev, p, stream);
}

}  // namespace

cudaError_t launch_w4a16_gemm(const W16Call &c, cudaStream_t stream) {
    W16Params p{};
    p.x = c.x;
    p.w = c.w;
    p.s = c.scales;
    p.y = c.y;
    p.M = c.M;
    p.N = c.N;
    p.K = c.K;
    p.ldx = c.ldx;
    p.out = c.out_type;
    p.grouped = c.group != c.K;
    switch (c.in_type) {
        case IN_F32: return launch_w16<IN_F32>(p, stream);
        case IN_BF16: return launch_w16<IN_BF16>(p, stream);
        default: return launch_w16<IN_F16>(p, stream);
    }
}

}  // namespace rq
