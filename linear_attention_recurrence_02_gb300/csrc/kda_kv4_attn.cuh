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

struct AttnArgs {
    const void *q;
    void *out;
    float *lse;       // or NULL
    float *part;      // pieces: [CTA][2][R rows][D], then [CTA][2][R][2] maxima and sums
    unsigned *err;
    Cache c;
    int64_t q_stride, out_stride;
    int Hq, group;    // query heads, and of one key/value head
    int causal, window;
    float scale_log2;  // scale * log2(e)
    int ctas;         // CTAs that cut the line
    int few_rows;     // > 0: sequences of more rows a key/value head are left to the other kernel; < 0: of at most -few_rows
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
    int64_t t0 = b, t1 = b + 1, len = a.c.lens[b];
    unsigned bad = 0;
    if (a.c.cu) {
        t0 = a.c.cu[b];
        t1 = a.c.cu[b + 1];
        if (t0 < 0 || t1 < t0 || t1 > a.c.T) {
            bad |= DEVERR_SEQLENS;
            t1 = t0 = 0;
        }
    }
    const int64_t most = (int64_t)a.c.cols << a.c.page_shift;
    if (len < 0 || len > most) {
        bad |= DEVERR_PAGES;
        len = len < 0 ? 0 : most;
    }
    if (bad && flag) atomicOr(a.err, bad);
    s.t0 = t0;
    s.n = (int)(t1 - t0);
    s.len = (int)len;
    const int rows = s.n * a.group;
    if (a.few_rows > 0 ? rows > a.few_rows : rows <= -a.few_rows) s.n = 0;
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
    const int64_t c = (total + ctas - 1) / ctas;
    return c < least ? least : c;
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
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        const unsigned past = __ballot_sync(0xffffffffu, before + upto > at);
        if (past) {
            const int l = __ffs(past) - 1;
            w.b = b0 + l;
            const int64_t rest = at - before - __shfl_sync(0xffffffffu, upto - mine, l);
            w.s = seq_at<R, TILE>(a, w.b, false);
            w.item = (int)(rest / w.s.tiles);
            w.t = (int)(rest - (int64_t)w.item * w.s.tiles);
            w.left = 0;
            return w;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    w.b = a.c.B;  // not reached
    w.item = w.t = 0;
    w.left = 0;
    w.s = Seq{0, 0, 0, 0, 1, 0};
    return w;
}

// What a run has of one item.
struct Segment {
    int64_t t0;         // the sequence's first new token
    int n, len;         // the sequence's new tokens and cached tokens
    int b, block, h;
    int first, last;    // tiles of the sequence that it covers and some row sees: [first, last)
    int piece;          // -1: the whole item, 0: it began in an earlier run, 1: it goes on in the next
};

template <int R, int TILE> __device__ __forceinline__ bool next_segment(const AttnArgs &a, Walk &w, Segment &g) {
    if (w.left <= 0) return false;
    while (w.item >= w.s.blocks * a.c.Hk) {
        if (++w.b >= a.c.B) return false;
        w.s = seq_at<R, TILE>(a, w.b, false);
        w.item = w.t = 0;
    }
    const int take = (int)min((int64_t)(w.s.tiles - w.t), w.left);
    g.t0 = w.s.t0;
    g.n = w.s.n;
    g.len = w.s.len;
    g.b = w.b;
    g.block = w.item / a.c.Hk;
    g.h = w.item - g.block * a.c.Hk;
    g.piece = w.t > 0 ? 0 : take < w.s.tiles ? 1 : -1;
    const int i0 = g.block * R / a.group, i1 = min(w.s.n * a.group - 1, g.block * R + R - 1) / a.group;
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
    return true;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Launches the kernel that joins the pieces of R rows each (tiles of TILE tokens, runs of at least `least`).
template <int D, typename T, int R, int TILE> kda_status launch_join(const AttnArgs &a, int least, cudaStream_t s);

}  // namespace kv4
}  // namespace kda
