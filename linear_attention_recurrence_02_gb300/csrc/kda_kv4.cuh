// kda_kv4.cuh -- the paged cache that holds keys and values in 4 bits: its format, and how a kernel
// quantises into it and expands from it.
//
// A group of 32 channels of one token shares a scale s, and code c in 1..15 stands for (c - 8) s:
//
//   s = max |x| / 7 rounded up to five significant bits,  c = 8 + x / s rounded to nearest
//
// Five bits, because (c - 8) s then has at most eight: every value the cache holds is a bf16 number, so
// the tensor cores take it without a rounding, and (16 + c) s - 24 s is one exact fused product. Rounded
// up, so that no value clips. The scale is a bf16 with its three lowest bits zero.
//
// A block of 18 D bytes holds 16 tokens of one key/value head, laid out for the fragments of a
// 16 x 8 x 16 matrix instruction, whose lanes (r, j) = (lane / 4, lane % 4) read
//
//   keys    [16 tokens][4 j][D/32 groups][4 bytes]   channels 32g + 8j + 0..7: operand rows are tokens
//   scales  [16 tokens][D/32]
//   values  [8 token pairs][8 r][2 tokens][D/32][2 bytes]  channels 32g + 8(r/2) + (r mod 2) + {0,2,4,6}:
//           operand rows are channels and pairs of tokens share a register. r stands at place
//           (r + 2 pair) mod 8, which keeps eight lanes' 16-byte reads on different banks
//   scales  [8 token pairs][D/32][2 tokens]
//
// Four bytes hold the even channels in their lower half and the odd ones in the upper; a half is its four
// codes, first lowest, rotated left by three bits. Bits 3..6 of a half are then the upper four of a bf16's
// seven mantissa bits: masked and joined to 16.0 they read 16 + c, two channels at once. The other three
// codes get there by a shift of four, a swap of bytes, and both.
#pragma once

#include "kda_common.cuh"

namespace kda {
namespace kv4 {

constexpr int BLOCK = 16;  // tokens of a block
constexpr float SCALE_MIN = 0x1p-100f, SCALE_MAX = 0x1p123f;

template <int D> struct Format {
    static constexpr int G = D / 32;       // groups of a token
    static constexpr int BYTES = 18 * D;   // of a block
    static constexpr int KS = 8 * D, V = 9 * D, VS = 17 * D;  // where key scales, values, value scales start
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }

// ---------------------------------------------------------------- expanding
// A word's eight codes as four pairs of bf16: f[i] = 16 + the codes of channels 2i and 2i + 1.
// `swapped` is the word with the bytes of each half exchanged. One of the two constants is hidden from the
// compiler, which otherwise puts both into instructions: an instruction holds one, so that masking and
// joining take two instead of one.
struct Expand {
    uint32_t base;
    __device__ __forceinline__ Expand() { asm volatile("mov.b32 %0, 0x41804180;" : "=r"(base)); }
    __device__ __forceinline__ uint32_t join(uint32_t x) const {
        uint32_t r;
        asm("lop3.b32 %0, %1, 0x00780078, %2, 0xea;" : "=r"(r) : "r"(x), "r"(base));  // (x & mask) | base
        return r;
    }
    __device__ __forceinline__ void codes16(uint32_t w, uint32_t swapped, uint32_t (&f)[4]) const {
        f[0] = join(w);
        f[1] = join(w >> 4);
        f[2] = join(swapped);
        f[3] = join(swapped >> 4);
    }
    __device__ __forceinline__ void operator()(uint32_t w, uint32_t swapped, uint32_t s2, uint32_t n2, uint32_t (&f)[4]) const;
};
__device__ __forceinline__ uint32_t swap_bytes(uint32_t w) { return prmt(w, 0, 0x2301); }

// (16 + c) s - 24 s, exact: 24 s has seven significant bits, the result at most eight.
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}
__device__ __forceinline__ uint32_t minus24(uint32_t s2) {
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(s2), "r"(0xC1C0C1C0u));
    return d;
}
__device__ __forceinline__ void Expand::operator()(uint32_t w, uint32_t swapped, uint32_t s2, uint32_t n2,
                                                   uint32_t (&f)[4]) const {
    codes16(w, swapped, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = fma_bf16x2(f[i], s2, n2);
}
__device__ __forceinline__ bool not_finite16(uint32_t bf16_bits) { return (bf16_bits & 0x7f80u) == 0x7f80u; }

// ---------------------------------------------------------------- quantising
// Maximum that a NaN wins.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
// A group's scale from its largest |x|: NaN where that is not finite.
__device__ __forceinline__ float group_scale(float m) {
    if (!(m < INFINITY)) return __uint_as_float(0x7fc00000u);
    // The smallest five-bit number with 7 s >= m (7 s is exact): m / 7 cut to five bits is at most two
    // steps below it, the second one where the product rounds below a number that m / 7 is just above.
    uint32_t b = __float_as_uint(m * (1.0f / 7.0f)) & ~0x7ffffu;
    if (7.0f * __uint_as_float(b) < m) b += 0x80000u;
    if (7.0f * __uint_as_float(b) < m) b += 0x80000u;
    return fminf(fmaxf(__uint_as_float(b), SCALE_MIN), SCALE_MAX);
}

constexpr uint32_t NAN_CODES = 0x44444444u;  // eight codes of 8, rotated
// Halves of four codes each (first lowest), the even channels' and the odd ones', as a word.
__device__ __forceinline__ uint32_t rotated(uint32_t even, uint32_t odd) {
    const uint32_t w = prmt(even, odd, 0x5410);
    return ((w << 3) & 0xfff8fff8u) | ((w >> 13) & 0x00070007u);
}
__device__ __forceinline__ void clip(float2 &x) {
    x = make_float2(fminf(fmaxf(x.x, -7.f * SCALE_MAX), 7.f * SCALE_MAX), fminf(fmaxf(x.y, -7.f * SCALE_MAX), 7.f * SCALE_MAX));
}

// Word of eight fp32 channels, as pairs of neighbours. The quotient is rounded as a division would round it: with the
// reciprocal correctly rounded, one residual step makes x * inv exact to the last bit (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990); values that lie between two codes
// are common, since inputs and scales have few bits. Adding 1.5 * 2^23 rounds to a whole number, halves to even;
// the four codes of a half are joined as whole numbers in fp32 (below 2^16, so exactly), two halves at once.
__device__ __forceinline__ uint32_t quantise8(float2 (&x)[4], float s) {
    if (!(s == s)) return NAN_CODES;
    if (s == SCALE_MAX) {
#pragma unroll
        for (int i = 0; i < 4; ++i) clip(x[i]);
    }
    const float inv = __frcp_rn(s);
    const float2 inv2 = make_float2(inv, inv), neg2 = make_float2(-s, -s);
    const float2 whole = make_float2(12582912.f, 12582912.f), less = make_float2(-12582912.f, -12582912.f);
    float2 code = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        float2 q = __fmul2_rn(x[i], inv2);
        q = __ffma2_rn(__ffma2_rn(q, neg2, x[i]), inv2, q);
        q = __fadd2_rn(__fadd2_rn(q, whole), less);
        code = __ffma2_rn(code, make_float2(16.f, 16.f), q);
    }
    // + 8 for every code, and 2^23 so that the number stands in the lowest bits
    code = __fadd2_rn(code, make_float2(8388608.f + 34952.f, 8388608.f + 34952.f));
    return rotated(__float_as_uint(code.x), __float_as_uint(code.y));
}

// The same for bf16 channels, which need no exact quotient: x has eight significant bits and s five, so that x / s is a
// code and a half or at least 1/512 away from one (|x - (k + 1/2) s| is a multiple of the smaller of x's last place and
// s / 64). x * inv with an approximate reciprocal, rounded to multiples of 2^-11 by adding 6144, is the half itself in
// the first case and on the same side of it in the second; the second sum rounds it to 8 + code, halves to even, in the
// lowest bits of 2^23 + 2^22. The codes are joined there as integers: what the four words have above 16 bits falls off.
__device__ __forceinline__ uint32_t quantise8_bf16(float2 (&x)[4], float s) {
    if (!(s == s)) return NAN_CODES;
    if (s == SCALE_MAX) {
#pragma unroll
        for (int i = 0; i < 4; ++i) clip(x[i]);
    }
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    const float2 inv2 = make_float2(inv, inv), fine = make_float2(6144.f, 6144.f);
    const float2 whole = make_float2(12582920.f - 6144.f, 12582920.f - 6144.f);
    uint32_t even = 0, odd = 0;
#pragma unroll
    for (int i = 3; i >= 0; --i) {
        const float2 c = __fadd2_rn(__ffma2_rn(x[i], inv2, fine), whole);
        even = even * 16 + __float_as_uint(c.x);
        odd = odd * 16 + __float_as_uint(c.y);
    }
    return rotated(even, odd);
}

// ---------------------------------------------------------------- places
// Byte of a block where word (g, j) of token t's keys starts, and the half r (of group g) of its values.
template <int D> __device__ __forceinline__ int key_at(int t, int j, int g) { return t * (D / 2) + j * (D / 8) + 4 * g; }
template <int D> __device__ __forceinline__ int value_at(int t, int r, int g) {
    constexpr int G = D / 32;
    const int p = t >> 1;
    return Format<D>::V + p * D + ((r + 2 * p) & 7) * (D / 8) + (t & 1) * (2 * G) + 2 * g;
}
template <int D> __device__ __forceinline__ int key_scale_at(int t, int g) { return Format<D>::KS + t * (D / 16) + 2 * g; }
template <int D> __device__ __forceinline__ int value_scale_at(int t, int g) {
    return Format<D>::VS + (t >> 1) * (D / 8) + 4 * g + 2 * (t & 1);
}

// A paged cache and the sequences in it.
struct Cache {
    uint8_t *data;
    const int32_t *table;   // [B][cols], page of every page_size tokens of a sequence
    const int64_t *lens;    // [B] tokens held, new ones included
    const int64_t *cu;      // [B + 1] new tokens of each sequence, or NULL: one each
    int64_t T;              // rows of the tensors with the new tokens
    int64_t table_stride;
    int B, Hk, pages, cols, page_shift;
};

// A sequence's new tokens [t0, t1) and its length, and what is wrong with them: bits of the device error word.
struct Range {
    int64_t t0, t1, len;
    unsigned bad;
};
__device__ __forceinline__ Range range_of(const Cache &c, int b) {
    Range r = {b, (int64_t)b + 1, c.lens[b], 0};
    if (c.cu) {
        r.t0 = c.cu[b];
        r.t1 = c.cu[b + 1];
        if (r.t0 < 0 || r.t1 < r.t0 || r.t1 > c.T) r.bad |= DEVERR_SEQLENS;
    }
    if (r.len < 0 || r.len > (int64_t)c.cols << c.page_shift) r.bad |= DEVERR_PAGES;
    return r;
}

// Of new token t: its sequence and its position there; false where it has none (rows behind the last
// sequence, before the beginning of one that counts fewer tokens than are new, of one that is wrong).
__device__ __forceinline__ bool token_place(const Cache &c, int64_t t, int &b, int64_t &pos) {
    b = (int)t;
    if (c.cu) {
        int lo = 0, hi = c.B;  // the last b with cu[b] <= t
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (c.cu[mid] <= t) lo = mid;
            else hi = mid;
        }
        b = lo;
    }
    const Range r = range_of(c, b);
    pos = r.len - (r.t1 - t);
    return r.bad == 0 && r.t0 <= t && t < r.t1 && pos >= 0;
}
// The page of position pos of sequence b, or -1 with the error word set.
__device__ __forceinline__ int page_of(const Cache &c, int b, int64_t pos, unsigned *err) {
    const int64_t col = pos >> c.page_shift;
    const int page = col < c.cols ? c.table[b * c.table_stride + col] : -1;
    if (page >= 0 && page < c.pages) return page;
    atomicOr(err, DEVERR_PAGES);
    return -1;
}

// Host: checks shared by the calls on a cache; fills `c`.
kda_status check_cache(const void *cache, const int32_t *table, const int64_t *lens, const int64_t *cu, int B,
                       int64_t T, int Hk, int D, int page_size, int64_t pages, int cols, int64_t table_stride,
                       kda_dtype dtype, Cache &c);

}  // namespace kv4
}  // namespace kda
