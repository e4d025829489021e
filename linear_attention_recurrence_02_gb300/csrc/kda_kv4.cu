// kda_kv4.cu -- keys and values written into the 4-bit cache and read back (kda_kv4_append, kda_kv4_read).
//
// Both are bound by memory: 2 or 4 bytes a channel on one side, 9/16 of a byte on the other. D / 8 lanes
// own a token of a head, eight channels each: a group's largest magnitude is two shuffles away, a token's
// keys of a head are one coalesced row of words. The halves that the value layout wants are exchanged
// between lanes of neighbouring groups, so that each lane moves one word there as well.
// Writing 22016 tokens of 8 heads of 128 in bf16 takes 25 us (4.6 TB/s; 28.8 with quotients as exact as fp32
// inputs need them; issue slots bound it, 72 % used, ALU 62 %), reading them back 19; fp32, twice the bytes, 44 and 43. Neighbouring tokens side by side in a warp, for whole lines of values, and the
// sequence found by 32 probes at once instead of by halving made no difference.
#include <string>

#include "kda_fp8.cuh"
#include "kda_kv4.cuh"
#include "kda_prefill.cuh"

namespace kda {
namespace kv4 {

constexpr int NT = 256;

// A group's largest magnitude, a NaN above all, and a lane's word of codes; all four lanes of the group call.
__device__ __forceinline__ float group_max(const Raw8<float> &r) {
    float f[8], m = 0.f;
    unpack8(r, f);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(f[e]));
    m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
    return max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
}
__device__ __forceinline__ float group_max(const Raw8<__nv_bfloat16> &r) {  // magnitudes in order as 16-bit integers
    const uint32_t k = 0x7fff7fffu;
    uint32_t m = __vmaxu2(__vmaxu2(r.v.x & k, r.v.y & k), __vmaxu2(r.v.z & k, r.v.w & k));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, 2));
    return __uint_as_float(max(m << 16, m & 0xffff0000u));
}
template <typename T> __device__ __forceinline__ uint32_t codes_of(const Raw8<T> &r, float s) {
    float f[8];
    unpack8(r, f);
    float2 x[4] = {make_float2(f[0], f[1]), make_float2(f[2], f[3]), make_float2(f[4], f[5]), make_float2(f[6], f[7])};
    if constexpr (sizeof(T) == 2) return quantise8_bf16(x, s);
    else return quantise8(x, s);
}

// A launch's first CTAs look at every sequence, for a wrong one may have no token: at CHECKED each. (The others' threads
// asked for one sequence each, 81393 tokens read in 82 us instead of 72.)
constexpr int CHECKED = 16 * NT;
__device__ __forceinline__ void check_sequences(const Cache &c, unsigned *err) {
    unsigned bad = 0;
    for (int b = blockIdx.x * CHECKED + threadIdx.x; b < c.B && b < (int)(blockIdx.x + 1) * CHECKED; b += NT) bad |= range_of(c, b).bad;
    if (bad) atomicOr(err, bad);
}

// HU heads a thread, a token's lookup (sequence, length, page) shared by them.
template <int D, typename T, int HU>
__global__ void __launch_bounds__(NT) kv4_append_kernel(const T *k, const T *v, Cache c, int64_t k_stride,
                                                        int64_t v_stride, int checks, unsigned *err) {
    constexpr int LPR = D / 8;  // lanes of a row
    const int hc = (c.Hk + HU - 1) / HU;
    const int64_t unit = ((int64_t)((int)blockIdx.x - checks) * NT + threadIdx.x) / LPR;
    const int64_t t = unit / hc;
    const int h0 = (int)(unit - t * hc) * HU, w = threadIdx.x % LPR, g = w >> 2, j = w & 3;
    dependent_launch();
    if ((int)blockIdx.x < checks) return check_sequences(c, err);
    Raw8<T> rk[HU] = {}, rv[HU] = {};
#pragma unroll
    for (int u = 0; u < HU; ++u)
        if (t < c.T && h0 + u < c.Hk) {
            load8(k + t * k_stride + (h0 + u) * D + 8 * w, rk[u]);
            load8(v + t * v_stride + (h0 + u) * D + 8 * w, rv[u]);
        }
    int b = 0, page = -1;
    int64_t pos = 0;
    if (t < c.T && token_place(c, t, b, pos)) page = page_of(c, b, pos, err);
    const int in_page = (int)(pos & ((1 << c.page_shift) - 1)), tt = in_page & (BLOCK - 1);
#pragma unroll
    for (int u = 0; u < HU; ++u) {
        const bool live = page >= 0 && h0 + u < c.Hk;
        uint32_t word[2], scale[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const Raw8<T> &raw = i == 0 ? rk[u] : rv[u];
            const float s = group_scale(group_max(raw));
            word[i] = codes_of<T>(raw, s);
            scale[i] = __float_as_uint(s) >> 16;
        }
        // lanes of groups 2a and 2a + 1 exchange halves: the first keeps r = 2j, the second r = 2j + 1
        const uint32_t got = __shfl_xor_sync(0xffffffffu, g & 1 ? word[1] & 0xffffu : word[1] >> 16, 4);
        const uint32_t vw = g & 1 ? got | (word[1] & 0xffff0000u) : (word[1] & 0xffffu) | (got << 16);
        if (!live) continue;
        uint8_t *blk = c.data + (((int64_t)page * c.Hk + h0 + u) << (c.page_shift - 4)) * Format<D>::BYTES +
                       (in_page >> 4) * Format<D>::BYTES;
        *reinterpret_cast<uint32_t *>(blk + key_at<D>(tt, j, g)) = word[0];
        *reinterpret_cast<uint32_t *>(blk + value_at<D>(tt, 2 * j + (g & 1), g & ~1)) = vw;
        if (j == 0) {
            *reinterpret_cast<uint16_t *>(blk + key_scale_at<D>(tt, g)) = (uint16_t)scale[0];
            *reinterpret_cast<uint16_t *>(blk + value_scale_at<D>(tt, g)) = (uint16_t)scale[1];
        }
    }
}

template <typename T> __device__ __forceinline__ void store_values(T *p, const uint32_t (&f)[4]);
template <> __device__ __forceinline__ void store_values(__nv_bfloat16 *p, const uint32_t (&f)[4]) {
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(f[0], f[1], f[2], f[3]));
}
template <> __device__ __forceinline__ void store_values(float *p, const uint32_t (&f)[4]) {
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(f[i] << 16);
        x[2 * i + 1] = __uint_as_float(f[i] & 0xffff0000u);
    }
    store8(p, x);
}

template <int D, typename T, int HU>
__global__ void __launch_bounds__(NT) kv4_read_kernel(Cache c, T *k, T *v, int64_t k_stride, int64_t v_stride,
                                                      int checks, unsigned *err) {
    constexpr int LPR = D / 8;
    const int hc = (c.Hk + HU - 1) / HU;
    const int64_t unit = ((int64_t)((int)blockIdx.x - checks) * NT + threadIdx.x) / LPR;
    const int64_t t = unit / hc;
    const int h0 = (int)(unit - t * hc) * HU, w = threadIdx.x % LPR, g = w >> 2, j = w & 3;
    dependent_launch();
    if ((int)blockIdx.x < checks) return check_sequences(c, err);
    int b = 0, page = -1;
    int64_t pos = 0;
    if (t < c.T && token_place(c, t, b, pos)) page = page_of(c, b, pos, err);
    const int in_page = (int)(pos & ((1 << c.page_shift) - 1)), tt = in_page & (BLOCK - 1);
    const Expand expand;
    uint32_t word[HU][2], scale[HU][2];
#pragma unroll
    for (int u = 0; u < HU; ++u) {
        word[u][0] = word[u][1] = scale[u][0] = scale[u][1] = 0;
        if (page >= 0 && h0 + u < c.Hk) {
            const uint8_t *blk = c.data + (((int64_t)page * c.Hk + h0 + u) << (c.page_shift - 4)) * Format<D>::BYTES +
                                 (in_page >> 4) * Format<D>::BYTES;
            word[u][0] = *reinterpret_cast<const uint32_t *>(blk + key_at<D>(tt, j, g));
            word[u][1] = *reinterpret_cast<const uint32_t *>(blk + value_at<D>(tt, 2 * j + (g & 1), g & ~1));
            scale[u][0] = *reinterpret_cast<const uint16_t *>(blk + key_scale_at<D>(tt, g));
            scale[u][1] = *reinterpret_cast<const uint16_t *>(blk + value_scale_at<D>(tt, g));
        }
    }
#pragma unroll
    for (int u = 0; u < HU; ++u) {
        // a lane of an even group holds r = 2j of its own and the next group, one of an odd group r = 2j + 1
        // of the group before and its own
        const uint32_t vw = word[u][1];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, g & 1 ? vw & 0xffffu : vw >> 16, 4);
        word[u][1] = g & 1 ? got | (vw & 0xffff0000u) : (vw & 0xffffu) | (got << 16);
        if (page < 0 || h0 + u >= c.Hk) continue;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t s2 = scale[u][i] * 0x10001u;
            uint32_t f[4];
            expand(word[u][i], swap_bytes(word[u][i]), s2, minus24(s2), f);
            store_values(i == 0 ? k + t * k_stride + (h0 + u) * D + 8 * w : v + t * v_stride + (h0 + u) * D + 8 * w, f);
        }
    }
}

static bool valid_page(int size) { return size >= BLOCK && size <= 256 && (size & (size - 1)) == 0; }

kda_status check_cache(const void *cache, const int32_t *table, const int64_t *lens, const int64_t *cu, int B,
                       int64_t T, int Hk, int D, int page_size, int64_t pages, int cols, int64_t table_stride,
                       kda_dtype dtype, Cache &c) {
    if (B < 0 || B > 1 << 30) return invalid("B must be in 0 .. 2^30");
    if (T < 0 || T > 0x7fffffffLL) return invalid("T must be in 0 .. 2^31 - 1");
    if (Hk < 1 || Hk > 32768) return invalid("Hk must be in 1 .. 32768");
    if (D != 64 && D != 128) return invalid("D must be 64 or 128");
    if (dtype != KDA_F32 && dtype != KDA_BF16) return invalid("dtype must be KDA_F32 or KDA_BF16");
    if (!valid_page(page_size))
        return invalid("page_size must be 16, 32, 64, 128 or 256");
    if (pages < 1 || pages > 0x7fffffffLL) return invalid("pages must be in 1 .. 2^31 - 1");
    if (cols < 1 || (int64_t)cols * page_size > 0x7fffff00LL)
        return invalid("the block table's columns times page_size must be in 1 .. 2^31 - 257");
    if (table_stride < cols && B > 1) return invalid("table_stride must be at least the block table's columns");
    if (cu == nullptr && T != B) return invalid("without cu_seqlens there must be one token for each sequence");
    if (cu != nullptr && B == 0 && T != 0) return invalid("tokens without a sequence");
    kda_status st;
    if (T > 0 && ((st = check_ptr(cache, "cache")) || (st = check_ptr(table, "block_table")) ||
                  (st = check_ptr(lens, "lens")) || (cu && (st = check_ptr(cu, "cu_seqlens")))))
        return st;
    int shift = 4;
    while ((1 << shift) < page_size) ++shift;
    c = Cache{static_cast<uint8_t *>(const_cast<void *>(cache)), table, lens, cu, T, table_stride, B, Hk, (int)pages,
              cols, shift};
    return KDA_OK;
}

// Token strides in elements: rows of Hk * D contiguous ones that start on 16 bytes.
static kda_status check_rows(const void *k, const void *v, int64_t k_stride, int64_t v_stride, const Cache &c, int D,
                             kda_dtype dtype) {
    kda_status st;
    if ((st = check_ptr(k, "k")) || (st = check_ptr(v, "v"))) return st;
    const int64_t row = (int64_t)c.Hk * D, unit = dtype == KDA_BF16 ? 8 : 4;
    if (c.T > 1 && (k_stride < row || v_stride < row)) return invalid("token strides must be at least Hk*D");
    if (c.T > 1 && (k_stride % unit || v_stride % unit)) return invalid("token strides must be multiples of 16 bytes");
    return KDA_OK;
}

// `most` heads a thread once that still leaves every SM its threads, one head a thread below that, for latency.
// bf16, 8 heads of 128: 22016 tokens written in 24.3 us with four, 25.7 with two, 32 with eight; 81393 read in 72 us
// with two, 78 with four, 90 with one.
constexpr int APPEND_HEADS = 4, READ_HEADS = 2;
template <typename F> static kda_status launch_rows(const Cache &c, int D, int most, F &&go) {
    const int hu = c.T * c.Hk * (D / 8) >= (int64_t)current_sms() * 2048 * 4 && c.Hk >= most ? most : 1;
    const int checks = (int)(((int64_t)c.B + CHECKED - 1) / CHECKED);
    const int64_t blocks = (c.T * ((c.Hk + hu - 1) / hu) * (D / 8) + NT - 1) / NT + checks;
    if (blocks > 0x7fffffffLL) return invalid("T*Hk*D too large for one launch");
    go((unsigned)blocks, checks, hu > 1);
    return KDA_OK;
}

template <int D, typename T>
static kda_status append(const void *k, const void *v, const Cache &c, int64_t ks, int64_t vs, unsigned *err,
                         cudaStream_t s) {
    const kda_status st = launch_rows(c, D, APPEND_HEADS, [&](unsigned blocks, int checks, bool several) {
        auto kern = several ? kv4_append_kernel<D, T, APPEND_HEADS> : kv4_append_kernel<D, T, 1>;
        launch_dependent(kern, dim3(blocks), dim3(NT), 0, s, static_cast<const T *>(k), static_cast<const T *>(v), c, ks,
                         vs, checks, err);
    });
    return st ? st : check_launch("kv4_append_kernel");
}
template <int D, typename T>
static kda_status read(const Cache &c, void *k, void *v, int64_t ks, int64_t vs, unsigned *err, cudaStream_t s) {
    const kda_status st = launch_rows(c, D, READ_HEADS, [&](unsigned blocks, int checks, bool several) {
        auto kern = several ? kv4_read_kernel<D, T, READ_HEADS> : kv4_read_kernel<D, T, 1>;
        launch_dependent(kern, dim3(blocks), dim3(NT), 0, s, c, static_cast<T *>(k), static_cast<T *>(v), ks, vs, checks, err);
    });
    return st ? st : check_launch("kv4_read_kernel");
}

}  // namespace kv4
}  // namespace kda

using namespace kda;

extern "C" size_t kda_kv4_cache_bytes(int64_t pages, int Hk, int page_size, int D) {
    if (pages < 0 || pages > 0x7fffffffLL || Hk < 1 || Hk > 32768 || !kv4::valid_page(page_size) || (D != 64 && D != 128)) return 0;
    return (size_t)pages * (size_t)Hk * (size_t)(page_size / 16) * 18u * (size_t)D;
}

extern "C" kda_status kda_kv4_append(const void *k, const void *v, void *cache, const int32_t *block_table,
                                     const int64_t *lens, const int64_t *cu_seqlens, int B, int64_t T, int Hk, int D,
                                     int page_size, int64_t pages, int table_cols, int64_t table_stride,
                                     int64_t k_stride, int64_t v_stride, kda_dtype dtype, kda_stream_t stream) {
    clear_detail();
    kv4::Cache c;
    kda_status st = kv4::check_cache(cache, block_table, lens, cu_seqlens, B, T, Hk, D, page_size, pages, table_cols,
                                     table_stride, dtype, c);
    if (st || T == 0) return st;
    if ((st = kv4::check_rows(k, v, k_stride, v_stride, c, D, dtype))) return st;
    if (cache == k || cache == v) return invalid("cache must not alias k or v");
    if ((st = bind_stream_device(stream))) return st;
    unsigned *err = device_error_word();
    if (!err) return fail(KDA_ERR_CUDA, "device error word unavailable");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == KDA_BF16)
        return D == 128 ? kv4::append<128, __nv_bfloat16>(k, v, c, k_stride, v_stride, err, s)
                        : kv4::append<64, __nv_bfloat16>(k, v, c, k_stride, v_stride, err, s);
    return D == 128 ? kv4::append<128, float>(k, v, c, k_stride, v_stride, err, s)
                    : kv4::append<64, float>(k, v, c, k_stride, v_stride, err, s);
}

extern "C" kda_status kda_kv4_read(const void *cache, const int32_t *block_table, const int64_t *lens,
                                   const int64_t *cu_seqlens, void *k, void *v, int B, int64_t T, int Hk, int D,
                                   int page_size, int64_t pages, int table_cols, int64_t table_stride,
                                   int64_t k_stride, int64_t v_stride, kda_dtype dtype, kda_stream_t stream) {
    clear_detail();
    kv4::Cache c;
    kda_status st = kv4::check_cache(cache, block_table, lens, cu_seqlens, B, T, Hk, D, page_size, pages, table_cols,
                                     table_stride, dtype, c);
    if (st || T == 0) return st;
    if ((st = kv4::check_rows(k, v, k_stride, v_stride, c, D, dtype))) return st;
    if (cache == k || cache == v || k == v) return invalid("k, v and cache must not alias one another");
    if ((st = bind_stream_device(stream))) return st;
    unsigned *err = device_error_word();
    if (!err) return fail(KDA_ERR_CUDA, "device error word unavailable");
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (dtype == KDA_BF16)
        return D == 128 ? kv4::read<128, __nv_bfloat16>(c, k, v, k_stride, v_stride, err, s)
                        : kv4::read<64, __nv_bfloat16>(c, k, v, k_stride, v_stride, err, s);
    return D == 128 ? kv4::read<128, float>(c, k, v, k_stride, v_stride, err, s)
                    : kv4::read<64, float>(c, k, v, k_stride, v_stride, err, s);
}
