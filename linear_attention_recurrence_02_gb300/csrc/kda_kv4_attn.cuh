// kda_kv4_attn.cuh -- what the kernels of kda_kv4_attention share: arguments and how the work is cut.
//
// An item is a block of R rows (new tokens of a sequence times the query heads of one key/value head) over
// that sequence's cached tokens. Items stand one behind the other in a line of tiles of TILE cached tokens,
// which the CTAs cut into equal runs: the lengths are known on the device only, and sequences of any
// lengths leave every CTA the same number of tiles. A run starts and ends inside an item as a rule. What
// it has of such an item goes to the workspace (at most two pieces a CTA: at its start and at its end), and
// a second kernel joins the pieces of each item in the order of the CTAs.
#pragma once

#include "kda_kv4.cuh"

namespace kda {
namespace kv4 {

// x / d for 0 <= x < 2^31 by a product with ceil(2^(31 + s) / d), 2^s >= d: a division costs some forty
// instructions, and an item needs a dozen.
struct Div {
    uint32_t mul, shift;
    Div() = default;
    __host__ explicit Div(uint32_t d) {
        shift = 0;
        while ((1u << shift) < d) ++shift;
        mul = (uint32_t)(((1ull << (31 + shift)) + d - 1) / d);
    }
    __device__ __forceinline__ int operator()(int x) const { return (int)(((uint64_t)(uint32_t)x * mul) >> (31 + shift)); }
};
__device__ __forceinline__ int64_t div64(int64_t x, int64_t d) {
    return ((x | d) >> 31) == 0 ? (int64_t)((uint32_t)x / (uint32_t)d) : x / d;
}

// What the second kernel needs of an item that a run leaves unfinished; pieces = 0: there is none.
struct Joint {
    int64_t t0;
    int n, block, h, pieces;
};

struct AttnArgs {
    const void *q;
    void *out;
    float *lse;       // or NULL
    float *part;      // pieces: [CTA][2][R rows][D]
    float2 *ml;       // their maxima and sums: [CTA][2][R]
    Joint *joint;     // [CTA]: the item that goes on behind its run, where that is the item's first piece
    unsigned *err;
    Cache c;
    int64_t q_stride, out_stride;
    int Hq, group;    // query heads, and of one key/value head
    Div by_group, by_hk;
    int causal, window;
    float scale_log2;  // scale * log2(e)
    int sms;          // of the stream's device
    int ctas;         // CTAs that cut the line
    int most_rows;    // sequences with more rows a key/value head are another kernel's
    int least_rows;   // and those with fewer
};

// A sequence as the items see it.
struct Seq {
    int64_t t0;        // its first new token
    int n, len;        // new tokens, cached tokens
    int lo_tile;       // first tile that any row sees
    int tiles, blocks; // tiles of an item (at least one), blocks of rows
};

template <int R, int TILE> __device__ __forceinline__ Seq seq_at(const AttnArgs &a, int b, bool flag) {
    Seq s;
    const Range r = range_of(a.c, b);
    if (r.bad && flag) atomicOr(a.err, r.bad);
    const bool none = r.bad & DEVERR_SEQLENS;
    const int64_t len = max((int64_t)0, min(r.len, (int64_t)a.c.cols << a.c.page_shift));
    s.t0 = r.t0;
    s.n = none ? 0 : (int)(r.t1 - r.t0);
    s.len = (int)len;
    const int rows = s.n * a.group;
    if (rows > a.most_rows || rows < a.least_rows) s.n = 0;
    const int64_t lo = a.window > 0 ? len - s.n - a.window + 1 : 0;
    s.lo_tile = lo > 0 ? (int)lo / TILE : 0;
    s.tiles = max((s.len + TILE - 1) / TILE - s.lo_tile, 1);
    s.blocks = (s.n * a.group + R - 1) / R;
    return s;
}

// All 32 lanes: tiles of the line, and its runs' length.
template <int R, int TILE> __device__ __forceinline__ int64_t line_tiles(const AttnArgs &a, int lane) {
    int64_t w = 0;
    for (int b = lane; b < a.c.B; b += 32) {
        const Seq s = seq_at<R, TILE>(a, b, blockIdx.x == 0);
        w += (int64_t)s.blocks * a.c.Hk * s.tiles;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
    return w;
}
// Below `least` tiles a run is not cut further: a CTA's warps have one each.
__device__ __forceinline__ int64_t run_length(int64_t total, int ctas, int least) {
    const int64_t c = div64(total + ctas - 1, ctas);
    return c < least ? least : c;
}

// All 32 lanes: the first lane up to whose end `at` is passed, counting from `before`, each lane with `mine`; `before` is then
// what stands ahead of it. Without such a lane -1, and `before` is what stands ahead of the next 32.
__device__ __forceinline__ int lane_past(int64_t mine, int64_t at, int lane, int64_t &before) {
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + upto > at);
    const int l = past ? __ffs(past) - 1 : -1;
    before += __shfl_sync(0xffffffffu, past ? upto - mine : upto, past ? l : 31);
    return l;
}

// A place in the line.
struct Walk {
    int64_t left;      // tiles left in the run
    int b, item, t;    // sequence, its item (block of rows * Hk + key/value head), tile of the item
    Seq s;
};

// All 32 lanes: the place of tile `at` (which exists).
template <int R, int TILE> __device__ __forceinline__ Walk walk_at(const AttnArgs &a, int64_t at, int lane) {
    Walk w;
    int64_t before = 0;
    for (int b0 = 0; b0 < a.c.B; b0 += 32) {
        int64_t mine = 0;
        if (b0 + lane < a.c.B) {
            const Seq s = seq_at<R, TILE>(a, b0 + lane, false);
            mine = (int64_t)s.blocks * a.c.Hk * s.tiles;
        }
        const int l = lane_past(mine, at, lane, before);
        if (l >= 0) {
            w.b = b0 + l;
            w.s = seq_at<R, TILE>(a, w.b, false);
            w.item = (int)div64(at - before, w.s.tiles);
            w.t = (int)(at - before - (int64_t)w.item * w.s.tiles);
            w.left = 0;
            return w;
        }
    }
    w.b = a.c.B;  // not reached
    w.item = w.t = 0;
    w.left = 0;
    w.s = Seq{0, 0, 0, 0, 1, 0};
    return w;
}

// All 32 lanes: the beginning of item `at`, left = 0; false where there are not so many. Reports the bad sequences on its
// way, and with `last` those behind it too, which may have no item.
template <int R, int TILE>
__device__ __forceinline__ bool item_at(const AttnArgs &a, int64_t at, int lane, bool last, Walk &w) {
    int64_t before = 0;
    for (int b0 = 0; b0 < a.c.B; b0 += 32) {
        int64_t mine = 0;
        if (b0 + lane < a.c.B) mine = (int64_t)seq_at<R, TILE>(a, b0 + lane, true).blocks * a.c.Hk;
        const int l = lane_past(mine, at, lane, before);
        if (l >= 0) {
            w.b = b0 + l;
            w.item = (int)(at - before);
            w.s = seq_at<R, TILE>(a, w.b, false);
            w.t = 0;
            w.left = 0;
            if (last)
                for (int b = b0 + 32 + lane; b < a.c.B; b += 32) seq_at<R, TILE>(a, b, true);
            return true;
        }
    }
    return false;
}

// Tiles of a block of rows where each block is cut by what its own rows see.
template <int R, int TILE>
__device__ __forceinline__ void block_tiles(const AttnArgs &a, int n, int len, int block, int &first, int &tiles) {
    const int i0 = a.by_group(block * R), i1 = a.by_group(min(n * a.group - 1, block * R + R - 1));
    const int hi = a.causal ? max(len - n + i1 + 1, 0) : len;
    const int lo = a.window > 0 ? max(len - n + i0 - a.window + 1, 0) : 0;
    first = lo / TILE;
    tiles = max((hi + TILE - 1) / TILE - first, 1);
}
// All lanes: the tiles of sequence b's items, each with COST more. A prompt of a million and a half tokens with 64 query
// heads on one key/value head has more than 2^31.
template <int R, int TILE, int COST>
__device__ __forceinline__ int64_t sequence_tiles(const AttnArgs &a, int b, int lane, bool flag) {
    const Seq s = seq_at<R, TILE>(a, b, flag);
    int64_t sum = 0;
    for (int k = lane; k < s.blocks; k += 32) {
        int first, tiles;
        block_tiles<R, TILE>(a, s.n, s.len, k, first, tiles);
        sum += tiles + COST;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum * a.c.Hk;
}

// What a run has of one item.
struct Segment {
    int64_t t0;         // the sequence's first new token
    int n, len;         // the sequence's new tokens and cached tokens
    int b, block, h;
    int first, last;    // tiles of the sequence that it covers and some row sees: [first, last)
    int piece;          // -1: the whole item, 0: it began in an earlier run, 1: it goes on in the next
    int rest;           // tiles that the item has behind this run
    bool there;         // false: the run has no more
};

template <int R, int TILE> __device__ __forceinline__ void next_segment(const AttnArgs &a, Walk &w, Segment &g) {
    g.there = false;
    if (w.left <= 0) return;
    while (w.item >= w.s.blocks * a.c.Hk) {
        if (++w.b >= a.c.B) return;
        w.s = seq_at<R, TILE>(a, w.b, false);
        w.item = w.t = 0;
    }
    const int take = (int)min((int64_t)(w.s.tiles - w.t), w.left);
    g.t0 = w.s.t0;
    g.n = w.s.n;
    g.len = w.s.len;
    g.b = w.b;
    g.block = a.by_hk(w.item);
    g.h = w.item - g.block * a.c.Hk;
    g.piece = w.t > 0 ? 0 : take < w.s.tiles ? 1 : -1;
    g.rest = w.s.tiles - w.t - take;
    const int i0 = a.by_group(g.block * R), i1 = a.by_group(min(w.s.n * a.group - 1, g.block * R + R - 1));
    const int hi = a.causal ? max(w.s.len - w.s.n + i1 + 1, 0) : w.s.len;
    const int lo = a.window > 0 ? max(w.s.len - w.s.n + i0 - a.window + 1, 0) : 0;
    g.first = max(w.s.lo_tile + w.t, lo / TILE);
    g.last = min(w.s.lo_tile + w.t + take, (hi + TILE - 1) / TILE);
    w.left -= take;
    w.t += take;
    if (w.t == w.s.tiles) {
        w.t = 0;
        ++w.item;
    }
    g.there = true;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// Pairs of fp32 as sums of bf16 pairs, as many as QS: one rounds (2^-8), two leave 2^-16, three hold all 24 bits.
template <int QS> __device__ __forceinline__ void split_bf16(float2 x, uint32_t (&p)[QS]) {
#pragma unroll
    for (int i = 0; i < QS; ++i) {
        p[i] = pack_bf16(x.x, x.y);
        if (i + 1 < QS)
            x = __ffma2_rn(make_float2(__uint_as_float(p[i] << 16), __uint_as_float(p[i] & 0xffff0000u)),
                           make_float2(-1.f, -1.f), x);
    }
}

// CTAs for `blocks` blocks of rows over Hk heads of at most `tiles` tiles: one for every `least` of them, at most `cap`.
inline int ctas_for(int64_t blocks, int Hk, int64_t tiles, int least, int cap) {
    const int64_t some = blocks < 1 << 20 ? blocks : 1 << 20;  // so that the product keeps within 64 bits
    const int64_t n = (some * Hk * tiles + least - 1) / least;
    return n < cap ? (int)n : cap;
}

// Bytes of the pieces of `ctas` runs of blocks of R rows, and where they stand in a workspace.
inline size_t pieces_bytes(int ctas, int R, int D) {
    return (size_t)ctas * (2 * (size_t)R * (D + 2) * sizeof(float) + sizeof(Joint));
}
inline void place_pieces(AttnArgs &a, void *workspace, int R, int D) {
    a.part = static_cast<float *>(workspace);
    a.ml = reinterpret_cast<float2 *>(a.part + (size_t)a.ctas * 2 * R * D);
    a.joint = reinterpret_cast<Joint *>(a.ml + (size_t)a.ctas * 2 * R);
}

// The kernel for many rows (bf16): blocks of 256 rows, tcgen05. Uses many_bytes(a.sms, D) of a.part.
kda_status attn_many(const AttnArgs &a, int D, cudaStream_t s);
inline size_t many_bytes(int sms, int D) { return pieces_bytes(sms, 256, D); }

// Launches the kernel that joins the pieces of items of R rows.
template <int D, typename T, int R> kda_status launch_join(const AttnArgs &a, cudaStream_t s);

}  // namespace kv4
}  // namespace kda
