// tree_device.cuh -- what the tree-attention kernels share: parameters, the
// schedule of tiles over CTAs, and where partial results lie.  Internal linkage.
//
// A unit is (sequence, KV head, block of ROWS query rows); its tokens are cut into
// tiles of TT.  All units form one line, each with its tiles and before them a lead
// that stands for its fixed cost, and CTA c of G takes the stretch [c T / G,
// (c + 1) T / G): CTAs end together whatever the lengths, long sequences spread over
// many of them, and a unit that lies inside one stretch is finished there.  A unit that
// spans CTAs leaves one partial per CTA: slot 2c for the unit the stretch begins in, 2c + 1
// for the last.
#pragma once

#include "paged_device.cuh"

#include <cmath>
#include <type_traits>

namespace rq {
namespace {

struct TreeParams {
    const void *q;
    int64_t q_token, q_head;            // strides in elements
    const uint8_t *kq, *vq;
    const float *ks, *vs;
    const int32_t *table, *contexts, *offsets;
    const uint8_t *mask;                // [rows][mask_stride], NULL: causal among the nodes
    int64_t mask_stride, width, pages, rows;
    int seqs, kv_heads, group, log_page, max_nodes;
    uint64_t seed;
    uint32_t flags;
    float score_scale;                  // softmax_scale * log2(e)
    float2 full_scale;                  // that by 1/sqrt(D), in two parts
    void *out;
    float *part;                        // [2 G][ROWS][D] fp32, then [2 G][ROWS][2] (reference, sum), then [G] TreeJoin
    int64_t rows_each;                  // query rows per KV head and sequence, on average
    int per_head;                       // blocks of rows per KV head and sequence that the join has blocks for; 0: see TreeJoin
    int ctas;                           // G
    int *err;
    static constexpr bool kPass = false;
};

// Where the pass over the prefixes has left a row's sums: as partials of its CTAs, as in TreeJoin;
// in the state, or nowhere.
struct alignas(8) TreePlace {
    uint32_t slots;                     // slot0, and the last CTA in the upper half
    int row;                            // of the block's
};
constexpr uint32_t kPlaceState = 0xffffffffu, kPlaceNone = 0xfffffffeu;

// One of two passes over a state (see TreePass): a unit that is finished leaves its rows there
// (out), or a unit's first tile begins with what they hold (in).
struct TreePassParams : TreeParams {
    const int32_t *groups;              // out: [seqs + 1] first sequences of the groups that are its sequences
    int group_seqs;
    float *state;
    float2 *state_ml;
    TreePlace *place;                   // NULL: a join between the passes leaves every row in the state
    const float *out_part;              // in: partials of the pass before, of blocks of so many rows, and its CTAs
    int out_rows, out_ctas;             // (out: set at its launch)
    bool out_pass;
    static constexpr bool kPass = true;
};

// Query rows per KV head and sequence on average: what the choice of a kernel goes by.  The
// bound max_nodes may be far above it (it is the number of rows where a caller has none).
inline int64_t tree_rows(const TreeCall &c) {
    const int64_t nodes = (c.rows + c.seqs - 1) / c.seqs;
    return (nodes < c.max_nodes ? nodes : c.max_nodes) * (c.q_heads / c.cache.heads);
}
// Host side: the parameters that do not depend on the kernel, and TMA maps whose boxes
// are whole pages, or a tile's worth of a larger page.
inline bool tree_params(const TreeCall &c, TreeParams &p) {
    p = TreeParams{};
    p.rows_each = tree_rows(c);
    p.q = c.q;
    p.q_token = c.q_token;
    p.q_head = c.q_head;
    p.kq = c.cache.kq;
    p.vq = c.cache.vq;
    p.ks = c.cache.ks;
    p.vs = c.cache.vs;
    p.table = c.table;
    p.contexts = c.contexts;
    p.offsets = c.offsets;
    p.mask = c.mask;
    p.mask_stride = c.mask_stride;
    p.width = c.width;
    p.rows = c.rows;
    p.pages = c.cache.pages;
    p.seqs = (int)c.seqs;
    p.kv_heads = (int)c.cache.heads;
    p.group = (int)(c.q_heads / c.cache.heads);
    while ((int64_t(1) << p.log_page) < c.cache.page_size) ++p.log_page;
    p.max_nodes = (int)c.max_nodes;
    p.seed = c.seed;
    p.flags = c.flags;
    p.score_scale = (float)((double)c.softmax_scale * 1.4426950408889634);
    const double full = (double)c.softmax_scale * 1.4426950408889634 / sqrt((double)c.head_dim);
    p.full_scale.x = (float)full;
    p.full_scale.y = (float)(full - (double)p.full_scale.x);
    p.out = c.out;
    p.part = static_cast<float *>(c.workspace);
    p.err = error_word_device_ptr();
    return p.err != nullptr;
}
inline bool tree_params(const TreePass &t, TreePassParams &p) {
    p = TreePassParams{};
    if (!tree_params(t.call, static_cast<TreeParams &>(p))) return false;
    p.groups = t.groups;
    p.group_seqs = (int)t.group_seqs;
    p.state = t.state;
    p.state_ml = reinterpret_cast<float2 *>(t.state + t.call.rows * t.call.q_heads * t.call.head_dim);
    p.place = static_cast<TreePlace *>(t.place);
    p.out_part = t.out_part;
    p.out_rows = t.out_rows;
    p.out_ctas = t.out_ctas;
    p.out_pass = t.groups != nullptr;
    return true;
}
inline bool tree_maps(const TreeCall &c, int tile, CUtensorMap &mk, CUtensorMap &mv) {
    const int64_t rows = c.cache.pages * c.cache.heads * c.cache.page_size;
    const int rb = (int)(c.head_dim / 2), box = (int)(c.cache.page_size < tile ? c.cache.page_size : tile);
    const CUtensorMapSwizzle sw = rb == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : rb == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                  : rb == 32 ? CU_TENSOR_MAP_SWIZZLE_32B
                                             : CU_TENSOR_MAP_SWIZZLE_NONE;
    return make_tma_map_u8(&mk, c.cache.kq, rows, rb, rb, box, sw) && make_tma_map_u8(&mv, c.cache.vq, rows, rb, rb, box, sw);
}

// At most so many tiles in all, with blocks of `block` rows: as far as the table reaches.
inline int64_t tree_tiles(const TreeCall &c, int64_t block, int64_t tile) {
    const int64_t group = c.q_heads / c.cache.heads, each = c.seqs * ((c.max_nodes * group + block - 1) / block),
                  all = c.seqs + c.rows * group / block;
    const double tiles = (double)(c.cache.heads * (each < all ? each : all)) * (double)((c.width * c.cache.page_size + tile - 1) / tile);
    return tiles < 1e9 ? (int64_t)tiles : 1000000000;
}

// log2 of a row's weights relative to its reference: where a move of the reference puts the
// largest, and past what the next move comes.  The products take weights as fp16, which
// holds 11 bits from 2^-14 to 2^16.  And log2 of the least value scale that the reference
// follows, so that the sum of the weights without their scales stays in range.
constexpr float kWeightTo = 9.f, kWeightMost = 15.f, kLeastValue = -60.f;

// The CTAs of a call, and whether the join goes by units: where there can be fewer of them.
inline void tree_ctas(const TreeCall &c, TreeParams &p, int64_t block, int64_t tile, int most) {
    const int64_t tiles = tree_tiles(c, block, tile), each = (c.max_nodes * p.group + block - 1) / block;
    p.ctas = (int)(tiles < most ? tiles : most);
    p.per_head = (double)c.seqs * p.kv_heads * each < p.ctas ? (int)each : 0;
}

struct TreeSeq {
    int64_t row0;      // first query row
    int ctx, n, len;   // tokens before the tree, nodes, tokens in all
    int mt, nt;        // row blocks, tiles
};

// The second of two passes may begin while the first still runs (its launch says so): nothing is
// handed on but the state, the rows' places and the partials.  Every thread of it waits for the
// first to end, before it reads those and at the latest before it exits: what follows on the
// stream is ordered behind the second pass alone.
__device__ __forceinline__ void pass_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Is this the pass over the groups' prefixes?
template <class P>
__device__ __forceinline__ bool out_pass(const P &p) {
    if constexpr (P::kPass) return p.out_pass;
    else return false;
}

template <int ROWS, int TT, class P>
__device__ __forceinline__ TreeSeq tree_seq(const P &p, int b) {
    TreeSeq s;
    int b0 = b, b1 = b + 1;
    if constexpr (P::kPass) {
        if (p.out_pass) {                                          // the rows of a group's sequences
            b0 = max(0, min(p.groups[b], p.group_seqs));
            b1 = max(0, min(p.groups[b + 1], p.group_seqs));
        }
    }
    const int64_t o0 = p.offsets[b0], o1 = min((int64_t)p.offsets[b1], p.rows);
    s.row0 = o0;
    s.n = o0 < 0 ? 0 : (int)max((int64_t)0, min(o1 - o0, (int64_t)p.max_nodes));
    const int64_t cap = p.width << p.log_page;
    s.ctx = (int)min((int64_t)max(0, p.contexts[b]), cap);         // what lies past the table is not seen
    s.len = out_pass(p) ? s.ctx : (int)min((int64_t)s.ctx + s.n, cap);
    s.mt = s.len ? (s.n * p.group + ROWS - 1) / ROWS : 0;          // no unit without a tile: the join goes by mt
    s.nt = s.mt ? (s.len + TT - 1) / TT : 0;
    return s;
}

// The state's place of row `r` of a row block.
template <int ROWS>
__device__ __forceinline__ int64_t tree_state(const TreeParams &p, int64_t row0, int mt, int h, int r) {
    const int gr = mt * ROWS + r;
    return ((row0 + gr / p.group) * p.kv_heads + h) * p.group + gr % p.group;
}

// Rows whose group has no prefix, or that belong to none, begin from nothing: what the pass over
// the prefixes leaves for them.  By all threads of its kernel.
template <int ROWS, int TT>
__device__ __forceinline__ void tree_clear(const TreePassParams &p) {
    const int64_t heads = (int64_t)p.kv_heads * p.group;
    auto clear = [&](int64_t r0, int64_t r1) {
        for (int64_t i = r0 * heads + threadIdx.x; i < r1 * heads; i += blockDim.x) {
            if (p.place) p.place[i] = TreePlace{kPlaceNone, 0};
            else p.state_ml[i] = make_float2(-INFINITY, 0.f);
        }
    };
    auto row = [&](int g) { return max((int64_t)0, min((int64_t)p.offsets[max(0, min(p.groups[g], p.group_seqs))], p.rows)); };
    if (blockIdx.x == 0) {
        clear(0, row(0));
        clear(row(p.seqs), p.rows);
    }
    for (int g = blockIdx.x; g < p.seqs; g += gridDim.x)
        if (tree_seq<ROWS, TT>(p, g).nt == 0) clear(row(g), row(g + 1));
}

constexpr int kScan = 128;              // stretches of sequences whose lengths are scanned

// The line of units: where each of kScan stretches of sequences begins and, at the end, its
// length; and the units' lead.
struct TreeLine {
    int64_t prefix[kScan + 1];
    int64_t units[kScan];
    int lead;
};

// What a unit costs a CTA beside its tiles, in tiles: q~, the first tile's latency, the
// masked tiles at its end and its output.  With tiles alone CTAs that meet several short
// units end last.  Measured: 0, 2, 4, 6 and 9 tiles give 87, 80, 77, 79 and 78 us for 16
// ragged sequences of up to 4k (128 rows, fp16), 105, 104, 103, 105 and 106 us for 64 of up
// to 8k (8 rows, bf16); 2 of 256k take 138 or 139 with any.  Less where CTAs have few tiles
// each: there the lead would leave some of them without any (one sequence of 512: 16 us
// without, 18 with 9).
__device__ __forceinline__ int tree_lead(int64_t tiles, int ctas) { return (int)(tiles / ctas < 8 ? tiles / ctas / 2 : 4); }

// In the passes of shared-prefix attention, whose units are many and short: blocks of few rows
// give a unit 10 tiles (2, 4, 6, 10, 16 and 28 give 424, 402, 384, 371, 373 and 378 us for
// 2048 units of up to 17 tiles, 456 CTAs), as far as CTAs are then left with half of their
// tiles (112 units of up to 24 tiles, 304 CTAs: 3, 5, 7 and 10 give 40.6, 37.0, 39.1 and 42.4).
template <int ROWS>
__device__ __forceinline__ int pass_lead(int64_t tiles, int64_t units, int ctas) {
    constexpr int most = ROWS >= 128 ? 4 : 10;
    return units >= ctas ? most : (int)min((int64_t)most, tiles / (ctas - units) / 2);
}

// A unit's length in the line: its tiles, and before them its lead.
__device__ __forceinline__ int64_t unit_length(int lead, const TreeSeq &s) { return s.nt ? s.nt + lead : 0; }

// Fills the line.  Every thread of the block calls it; ends with a block barrier.
template <int ROWS, int TT, class P>
__device__ __forceinline__ void tree_scan(const P &p, TreeLine &line) {
    const int per = (p.seqs + kScan - 1) / kScan;
    if (threadIdx.x < kScan) {
        int64_t tiles = 0, units = 0;
        for (int b = threadIdx.x * per; b < min(p.seqs, ((int)threadIdx.x + 1) * per); ++b) {
            const TreeSeq s = tree_seq<ROWS, TT>(p, b);
            tiles += (int64_t)p.kv_heads * s.mt * s.nt;
            units += s.nt ? (int64_t)p.kv_heads * s.mt : 0;
        }
        line.prefix[threadIdx.x] = tiles;
        line.units[threadIdx.x] = units;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        int64_t v[kScan / 32], u[kScan / 32], tiles = 0, units = 0;
#pragma unroll
        for (int i = 0; i < kScan / 32; ++i) {
            v[i] = line.prefix[threadIdx.x * (kScan / 32) + i];
            u[i] = line.units[threadIdx.x * (kScan / 32) + i];
            tiles += v[i];
            units += u[i];
        }
        int64_t all = tiles;
#pragma unroll
        for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
        int lead;
        if constexpr (P::kPass) {
            int64_t of = units;
#pragma unroll
            for (int o = 16; o; o >>= 1) of += __shfl_xor_sync(0xffffffffu, of, o);
            lead = pass_lead<ROWS>(all, of, p.ctas);
        } else {
            lead = tree_lead(all, p.ctas);
        }
        const int64_t run = tiles + lead * units;
        int64_t incl = run;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
            if (threadIdx.x >= o) incl += x;
        }
        int64_t at = incl - run;
#pragma unroll
        for (int i = 0; i < kScan / 32; ++i) {
            line.prefix[threadIdx.x * (kScan / 32) + i] = at;
            at += v[i] + lead * u[i];
        }
        if (threadIdx.x == 31) line.prefix[kScan] = at;
        if (threadIdx.x == 0) line.lead = lead;
    }
    __syncthreads();
}

// Tiles that one accumulator adds up.  The tensor cores do not round their additions to
// nearest: sums of a common sign lose about 2^-24 of themselves with each, 256 tiles of 8
// additions 6e-5, as the sum grows meanwhile.  2048 tiles in one sum were 2e-4 (few rows) to
// 1.5e-3 (256 rows) off; fp16 is 2e-5 off now.
constexpr int kPieceTiles = 256;

// A piece of a CTA's stretch of a unit: all of it, or so many tiles.  What the pieces before
// have summed waits where the stretch's partial goes.
struct TreeWork {
    TreeSeq s;
    int b, h, mt;          // sequence, KV head, row block
    int t0, t1;            // the piece's tiles; none where the stretch ends within the unit's lead
    int64_t first, used;   // where the unit begins in the line; the piece's length
    bool begins;           // the stretch's first piece
    bool whole;            // the unit lies in this CTA alone, and this is its last piece
};

template <int ROWS, int TT, class P>
__device__ __forceinline__ TreeWork tree_work(const P &p, const TreeLine &line, int64_t pos, int64_t begin, int64_t end) {
    int lo = 0, hi = kScan;
    while (hi - lo > 1) {                    // the last stretch that begins at or before pos
        const int mid = (lo + hi) >> 1;
        if (line.prefix[mid] <= pos) lo = mid;
        else hi = mid;
    }
    const int per = (p.seqs + kScan - 1) / kScan;
    int64_t at = line.prefix[lo];
    TreeWork w;
    w.b = lo * per;
    while (true) {
        w.s = tree_seq<ROWS, TT>(p, w.b);
        const int64_t length = (int64_t)p.kv_heads * w.s.mt * unit_length(line.lead, w.s);
        if (pos < at + length || w.b + 1 >= p.seqs) break;
        at += length;
        ++w.b;
    }
    const int64_t off = pos - at, length = unit_length(line.lead, w.s), u = off / length, from = off - u * length;
    w.first = pos - from;
    w.begins = from == 0 || pos == begin;
    w.t0 = (int)max((int64_t)0, from - line.lead);
    w.used = min(min(length - from, end - pos), w.t0 + kPieceTiles + line.lead - from);
    w.t1 = (int)max((int64_t)0, from + w.used - line.lead);
    w.h = (int)(u / w.s.mt);
    w.mt = (int)(u - (int64_t)w.h * w.s.mt);
    w.whole = begin - w.first <= line.lead && w.t1 == w.s.nt;
    return w;
}

__device__ __forceinline__ int64_t tree_begin(int64_t total, int ctas, int c) { return total * c / ctas; }

// What the join has to know of a unit that spans CTAs; the CTA with its first tile leaves it,
// the others (and that one for none) one without rows.  The join has neither scan nor search,
// and as many blocks as CTAs, however many units there are; or, where there can be fewer
// units than CTAs, as many as units (p.per_head > 0), each with a place of its own.
struct alignas(16) TreeJoin {
    int row0, rows, h, mt; // the unit's first query row, its rows, KV head, row block
    int c1, slot0;         // its last CTA; the slot of the first CTA's partial, 2 c0 or one more
    int64_t total;         // the line's length
};
// floats before the TreeJoin of CTA 0
__host__ __device__ inline int64_t tree_join_at(int ctas, int rows, int dim) { return (int64_t)2 * ctas * rows * (dim + 2); }

template <int ROWS, int D>
__device__ __forceinline__ TreeJoin *tree_joins(const TreeParams &p) { return reinterpret_cast<TreeJoin *>(p.part + tree_join_at(p.ctas, ROWS, D)); }

// The slot of a stretch's partial.
__device__ __forceinline__ int tree_slot(const TreeWork &w, int64_t begin) { return 2 * (int)blockIdx.x + (begin >= w.first ? 0 : 1); }

// After each of a CTA's pieces (`join` begins as {}), when its loads are on their way: notes a
// unit that goes on past the CTA.
template <int ROWS, int D>
__device__ __forceinline__ void tree_note(const TreeParams &p, const TreeLine &line, const TreeWork &w, int64_t begin, int64_t end, TreeJoin &join) {
    if (w.t0 != 0 || w.t1 == 0) return;
    const int64_t total = line.prefix[kScan], last = w.first + unit_length(line.lead, w.s) - 1;
    if (last >= end) {
        // CTA of a position: the last c with total c / ctas <= position
        const int c1 = (int)(((last + 1) * p.ctas - 1) / total);
        join = TreeJoin{(int)w.s.row0, min(ROWS, w.s.n * p.group - w.mt * ROWS), w.h, w.mt, c1,
                        tree_slot(w, begin), total};
    }
    if (p.per_head && (threadIdx.x & 31) == 0)              // that of a unit that ends here is {}
        tree_joins<ROWS, D>(p)[((int64_t)w.b * p.kv_heads + w.h) * p.per_head + w.mt] = join;
}
// At the end of the CTA.
template <int ROWS, int D>
__device__ __forceinline__ void tree_noted(const TreeParams &p, const TreeJoin &join) {
    if (!p.per_head && (threadIdx.x & 31) == 0) tree_joins<ROWS, D>(p)[blockIdx.x] = join;
}

// Instead of the join's notes, in the pass over the prefixes: where the pass after it finds the unit's rows.
template <int ROWS>
__device__ __forceinline__ void tree_place(const TreePassParams &p, const TreeLine &line, const TreeWork &w, int64_t begin, int64_t end) {
    if (w.t0 != 0 || w.t1 == 0) return;
    const int64_t total = line.prefix[kScan], last = w.first + unit_length(line.lead, w.s) - 1;
    uint32_t slots = kPlaceState;
    if (last >= end) slots = (uint32_t)tree_slot(w, begin) | (uint32_t)(((last + 1) * p.ctas - 1) / total) << 16;
    const int rows = min(ROWS, w.s.n * p.group - w.mt * ROWS);
    for (int r = threadIdx.x & 31; r < rows; r += 32) p.place[tree_state<ROWS>(p, w.s.row0, w.mt, w.h, r)] = TreePlace{slots, r};
}

// A CTA of that pass without a stretch, where there are more CTAs than tiles: its partials are empty.
template <int ROWS, int D>
__device__ __forceinline__ void tree_empty(const TreePassParams &p) {
    if (!p.out_pass || !p.place) return;
    float2 *const ml = reinterpret_cast<float2 *>(p.part + (int64_t)2 * p.ctas * ROWS * D) + (int64_t)2 * blockIdx.x * ROWS;
    for (int r = threadIdx.x; r < ROWS; r += blockDim.x) ml[r] = make_float2(-INFINITY, 0.f);
}

// What a row's sums are to be joined with: n pairs (reference, sum) at ml + k ml_step, the lane's E
// dims at from + k step; the first of them by itself.
struct TreeBefore {
    const float2 *ml, *ml0;
    const float *from, *from0;
    int64_t ml_step, step;
    int n;
};
template <int D>
__device__ __forceinline__ TreeBefore tree_before(const TreePassParams &p, int64_t at) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const TreePlace u = p.place[at];
    if (u.slots == kPlaceState) return TreeBefore{p.state_ml + at, p.state_ml + at, p.state + at * D + lane * E, p.state + at * D + lane * E, 0, 0, 1};
    // within the scratch, whatever groups and offsets that are not in order have left unwritten
    const int R = p.out_rows, slot0 = min((int)(u.slots & 0xffffu), 2 * p.out_ctas - 1), c0 = slot0 >> 1,
              c1 = min((int)(u.slots >> 16), p.out_ctas - 1), row = max(0, min(u.row, R - 1));
    const float2 *const ml = reinterpret_cast<const float2 *>(p.out_part + (int64_t)2 * p.out_ctas * R * D) + row;
    // blocks of 128 rows and more leave pieces of 4 dims, [D / 4][R]
    const float *const from = p.out_part + (R >= 128 ? (lane * E / 4 * R + row) * 4 + (lane * E & 3) : row * D + lane * E);
    return TreeBefore{ml + (int64_t)2 * c0 * R, ml + (int64_t)slot0 * R, from + (int64_t)2 * c0 * R * D, from + (int64_t)slot0 * R * D,
                      (int64_t)2 * R, (int64_t)2 * R * D, u.slots == kPlaceNone ? 0 : c1 - c0 + 1};
}
// By a warp: a row's reference, sum and dims with those before them, in their order.  Few
// instructions, as each is fetched for the first time here: a version for all rows of a warp at
// once took 25 us for 20 (4 sequences), 84 for 60 (64 sequences).
template <int E>
__device__ __forceinline__ void tree_onto(const TreeBefore &b, float &top, float &sum, float (&acc)[E]) {
    constexpr int V = E < 4 ? E : 4, KS = 4;                // partials at a time
    using Vec = typename std::conditional<V == 4, float4, typename std::conditional<V == 2, float2, float>::type>::type;
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int base = 0; base < b.n; base += 32) {
        const int k = base + lane;
        const float2 x = k < b.n ? (k ? b.ml[k * b.ml_step] : *b.ml0) : make_float2(-INFINITY, 0.f);
        float t = fmaxf(top, x.x);
#pragma unroll
        for (int o = 16; o; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
        const float f = x.x == -INFINITY ? 0.f : ex2(x.x - t), g = top == -INFINITY ? 0.f : ex2(top - t);
        float add = f == 0.f ? 0.f : x.y * f;               // an empty partial adds nothing
#pragma unroll
        for (int o = 16; o; o >>= 1) add += __shfl_xor_sync(0xffffffffu, add, o);
        top = t;
        sum = (g == 0.f ? 0.f : sum * g) + add;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = g == 0.f ? 0.f : acc[e] * g;
#pragma unroll 1
        for (int k0 = 0; k0 < min(32, b.n - base); k0 += KS) {
            Vec y[KS][E / V];
            float fk[KS];
#pragma unroll
            for (int j = 0; j < KS; ++j) {
                fk[j] = __shfl_sync(0xffffffffu, f, k0 + j);                     // 0: nothing there to read
                const int kk = base + k0 + j;
                const float *from = kk ? b.from + kk * b.step : b.from0;
#pragma unroll
                for (int v = 0; v < E / V; ++v) y[j][v] = fk[j] != 0.f ? *reinterpret_cast<const Vec *>(from + v * V) : Vec{};
            }
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int e = 0; e < E; ++e) acc[e] += fk[j] * reinterpret_cast<const float *>(&y[j][e / V])[e % V];
        }
    }
}

// May query row `r` of the row block see token `t` of the sequence?  Rows past the
// sequence's last see nothing.
template <int ROWS>
__device__ __forceinline__ bool tree_sees(const TreeParams &p, const TreeWork &w, int r, int t) {
    const int i = (w.mt * ROWS + r) / p.group;
    if (i >= w.s.n || t >= w.s.len) return false;
    if (t < w.s.ctx) return true;
    const int j = t - w.s.ctx;
    return p.mask ? p.mask[(w.s.row0 + i) * p.mask_stride + j] != 0 : j <= i;
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t t_smem(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ void t_mbar_init(uint64_t *b, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(t_smem(b)), "r"(count) : "memory");
}
__device__ __forceinline__ void t_mbar_arrive(uint64_t *b) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(t_smem(b)) : "memory");
}
__device__ __forceinline__ void t_mbar_expect(uint64_t *b, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(t_smem(b)), "r"(bytes)
                 : "memory");
}
// The hint lets the hardware suspend the thread for up to 20 us: waiting warps then
// leave their issue slots to the others.
__device__ __forceinline__ bool t_mbar_try(uint64_t *b, uint32_t parity) {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2, %3;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(ok) : "r"(t_smem(b)), "r"(parity), "r"(20000u) : "memory");
    return ok != 0;
}
constexpr long long kTreeWaitLimit = 4000000000ll;   // ~2 s at 2 GHz

// Bounded wait.  On expiry it raises the error word and the CTA's abort flag; the
// caller goes on through its loops (whose later waits return at once), so that
// barriers between warps still meet.
// PASS: what is waited for may stand behind warps that are in pass_wait, for as long as the first
// of two passes takes.  A wait that has run out then stands behind the first pass too, and counts
// anew from its end (in the first pass nothing is before it).  The warps that go on
// from the first pass have none of these: they meet at a barrier of theirs before their next wait.
template <bool PASS>
__device__ __forceinline__ bool t_mbar_wait(uint64_t *b, uint32_t parity, volatile int *abort_flag, int *err) {
    if (t_mbar_try(b, parity)) return true;
    long long limit = (clock64() + kTreeWaitLimit) & -2ll;         // even: the first count
    while (true) {
        if (t_mbar_try(b, parity)) return true;
        if (*abort_flag) return false;
        if (clock64() > limit) {
            if (PASS && !(limit & 1)) {
                pass_wait();
                limit = (clock64() + kTreeWaitLimit) | 1ll;
                continue;
            }
            *abort_flag = 1;
            atomicExch(err, 1);
            return false;
        }
    }
}

__device__ __forceinline__ void t_tma_2d(void *dst, const CUtensorMap *map, uint64_t *bar, int y) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            t_smem(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(y), "r"(t_smem(bar))
        : "memory");
}
__device__ __forceinline__ void t_bulk(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     t_smem(dst)),
                 "l"(src), "r"(bytes), "r"(t_smem(bar))
                 : "memory");
}

// Joins the partials of the units that span CTAs: per row, in the order of the
// CTAs (so results do not change from run to run), the largest reference, the
// rescaled sums, then normalisation, R^T and the one rounding to the output type.
// Block c takes the unit whose first tile CTA c has (or unit c), if that spans CTAs.  A warp
// takes a row (two of 256-row units) and four partials at a time, so that their loads
// overlap.
// Launched so that it may begin while the kernel before it ends.  Every thread waits for
// that, those without a unit to join too: the join may not end before the kernel before it
// has, as what follows on the stream (or in a captured graph) is ordered behind the join
// alone.
__device__ __forceinline__ void tree_join_may_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
constexpr int join_rows(int rows) { return rows >= 256 ? 2 : 1; }         // rows per warp
constexpr int join_warps(int rows) { return rows < 16 ? rows : 16; }
constexpr int kJoinPerSm = 2;          // blocks: three leave registers for fewer loads at once (16 sequences of up to 4k: 76 us for 72)
template <int IN, int D, int ROWS, class P>
__global__ void __launch_bounds__(32 * join_warps(ROWS), kJoinPerSm) attn_tree_join_kernel(const __grid_constant__ P p, int turns) {
    constexpr int E = D / 32, RW = join_rows(ROWS), kJoinWarps = join_warps(ROWS);
    if (out_pass(p)) tree_join_may_begin();                 // here: the second pass
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int begin_row = (blockIdx.y * turns * kJoinWarps + warp) * RW;
    bool there_is = true;                                   // unit c, if blocks have units: its notes are old where it is not
    if (p.per_head) {
        const int b = blockIdx.x / (p.kv_heads * p.per_head);
        there_is = (int)(blockIdx.x % p.per_head) < tree_seq<ROWS, 128>(p, b).mt;
    }
    float sg[E];
    lane_signs<E>(sg, lane, p.seed);
    asm volatile("griddepcontrol.wait;" ::: "memory");      // the partials are written
    TreeJoin u{};
    if (there_is) u = tree_joins<ROWS, D>(p)[blockIdx.x];
    const int rows = u.rows, c0 = u.slot0 >> 1, c1 = u.c1;
    if (begin_row >= rows) return;
    const int64_t total = u.total;
    const float *ml = p.part + (int64_t)2 * p.ctas * ROWS * D;
    auto there = [&](int c) { return c <= c1 && tree_begin(total, p.ctas, c) != tree_begin(total, p.ctas, c + 1); };   // no empty stretch
    auto slot = [&](int c) { return (int64_t)(c == c0 ? u.slot0 : 2 * c); };
    for (int turn = 0; turn < turns; ++turn) {
    const int row0 = begin_row + turn * kJoinWarps * RW;
    if (row0 >= rows) break;
    float top[RW], sum[RW], acc[RW][E];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        top[i] = -INFINITY;
        sum[i] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[i][e] = 0.f;
    }
    for (int c = c0 + lane; c <= c1; c += 32) {
        if (!there(c)) continue;
        const float2 *x = reinterpret_cast<const float2 *>(ml) + slot(c) * ROWS + row0;
#pragma unroll
        for (int i = 0; i < RW; ++i)
            if (row0 + i < rows) top[i] = fmaxf(top[i], x[i].x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < RW; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
    for (int base = c0; base <= c1; base += 32) {
        const int c = base + lane;
        const bool on = there(c);
        const int64_t sl = on ? slot(c) : 0;
        float f[RW];
#pragma unroll
        for (int i = 0; i < RW; ++i) {
            f[i] = 0.f;
            if (on && row0 + i < rows) {
                const float2 x = reinterpret_cast<const float2 *>(ml)[sl * ROWS + row0 + i];
                if (x.x != -INFINITY) {                     // an empty partial adds nothing
                    f[i] = ex2(x.x - top[i]);
                    sum[i] += x.y * f[i];
                }
            }
        }
        for (int k0 = 0; k0 < min(32, c1 - base + 1); k0 += 4) {
            float x[4][RW][E], fk[4][RW];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float *a = p.part + (__shfl_sync(0xffffffffu, sl, k0 + k) * ROWS + row0) * D + lane * E;
#pragma unroll
                for (int i = 0; i < RW; ++i) {
                    fk[k][i] = __shfl_sync(0xffffffffu, f[i], k0 + k);       // 0: nothing there to read
#pragma unroll
                    for (int e = 0; e < E; ++e) x[k][i][e] = fk[k][i] != 0.f ? a[i * D + e] : 0.f;
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < RW; ++i)
#pragma unroll
                    for (int e = 0; e < E; ++e) acc[i][e] += fk[k][i] * x[k][i][e];
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < RW; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    if constexpr (P::kPass) {
        if (p.out_pass) {
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                if (row0 + i >= rows) break;
                const int64_t at = tree_state<ROWS>(p, u.row0, u.mt, u.h, row0 + i);
#pragma unroll
                for (int e = 0; e < E; ++e) p.state[at * D + lane * E + e] = acc[i][e];
                if (lane == 0) p.state_ml[at] = make_float2(top[i], sum[i]);
            }
            continue;
        }
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const float il = sum[i] == 0.f ? 0.f : 1.f / sum[i];    // nothing visible: zeros
#pragma unroll
        for (int e = 0; e < E; ++e) acc[i][e] *= il;
    }
    if (!(p.flags & RQ_ATTN_ROTATED_OUT)) {
#pragma unroll
        for (int i = 0; i < RW; ++i) warp_rotate<E>(acc[i], sg, lane, !(p.flags & RQ_SIGNS_FIRST), inv_sqrt_dim<D>());
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const int gr = u.mt * ROWS + row0 + i;
        if (row0 + i >= rows) break;
        const int64_t at = (((int64_t)u.row0 + gr / p.group) * p.kv_heads + u.h) * p.group + gr % p.group;
#pragma unroll
        for (int e = 0; e < E; ++e) store_elem<IN>(p.out, at * D + lane * E + e, acc[i][e]);
    }
    }
}

// Launches a kernel of the schedule: the second of two passes beside the end of the first.
template <class P, class... Args>
cudaError_t launch_tree_kernel(void (*kern)(Args...), const P &p, int threads, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.ctas);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    if constexpr (P::kPass) cfg.numAttrs = p.out_pass ? 0 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// Does every unit lie in one CTA, as there is but one, or no sequence can pass a tile?  Then there
// is nothing to join (4 sequences with a prompt of 1000 and 37 own tokens: 19.6 to 17.8 us).
inline bool tree_whole(const TreeParams &p) { return p.ctas == 1 || p.width << p.log_page <= 128; }

template <int IN, int D, int ROWS, class P>
cudaError_t launch_tree_join(const P &p, cudaStream_t stream) {
    if (tree_whole(p)) return cudaSuccess;
    const int blocks = p.per_head ? p.seqs * p.kv_heads * p.per_head : p.ctas - 1;
    // one turn per block while the SMs hold them all, counting the rows that there are on
    // average; then blocks take several
    constexpr int rows = join_warps(ROWS) * join_rows(ROWS);
    const int64_t filled = p.rows_each < ROWS ? p.rows_each : ROWS;
    int turns = 1;
    while (turns * rows < filled && blocks * ((filled + turns * rows - 1) / (turns * rows)) > kJoinPerSm * device_sm_count()) turns *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (ROWS + turns * rows - 1) / (turns * rows));
    cfg.blockDim = dim3(32 * join_warps(ROWS));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_tree_join_kernel<IN, D, ROWS, P>, p, turns);
}

}  // namespace
}  // namespace rq
