// fa_paged.cuh -- the paged KV cache's kernels: append (rotation by position, 16-bit or
// 4-bit pages) and read-back.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/fa.h"
#include "sm100.cuh"

namespace fa {

// Device status of these kernels: [0] fa_status code of the first failure, [1] the call.
static __device__ uint32_t g_paged_status[4];

enum : uint32_t { PAGED_APPEND = 0x401, PAGED_GATHER, PAGED_FWD };

__device__ __forceinline__ void record_bad_page(uint32_t where)
{
    if (atomicCAS(&g_paged_status[0], 0u, static_cast<uint32_t>(FA_ERR_BAD_PAGE)) == 0u) g_paged_status[1] = where;
}

// ---------------------------------------------------------------------------------
// 16-bit values: two per 32-bit word, the first in the low half.
// ---------------------------------------------------------------------------------
template <bool BF16>
__device__ __forceinline__ uint32_t pg_pack2(float lo, float hi)
{
    if constexpr (BF16) {
        __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&v);
    } else {
        __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<uint32_t*>(&v);
    }
}
template <bool BF16>
__device__ __forceinline__ float2 pg_unpack2(uint32_t w)
{
    if constexpr (BF16) return __bfloat1622float2(*reinterpret_cast<__nv_bfloat162*>(&w));
    else return __half22float2(*reinterpret_cast<__half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ void pg_unpack8(const uint4& w, float (&x)[8])
{
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = pg_unpack2<BF16>(u[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}
template <bool BF16>
__device__ __forceinline__ uint4 pg_pack8(const float (&x)[8])
{
    return make_uint4(pg_pack2<BF16>(x[0], x[1]), pg_pack2<BF16>(x[2], x[3]), pg_pack2<BF16>(x[4], x[5]),
                      pg_pack2<BF16>(x[6], x[7]));
}

// ---------------------------------------------------------------------------------
// The pools.  A (page, head) block is page_size rows of d 16-bit values, or page_size
// rows of d / 2 code bytes followed by page_size rows of d / 32 (scale, zero) pairs.
// ---------------------------------------------------------------------------------
struct PoolView {
    const int* table;  // [B, max_pages]
    int Hkv, page_size, page_shift, num_pages, max_pages;
};

template <int D, bool INT4>
__device__ __forceinline__ size_t pool_block_bytes(const PoolView& v)
{
    return static_cast<size_t>(v.page_size) * (INT4 ? 5 * D / 8 : 2 * D);
}
template <int D, bool INT4>
__device__ __forceinline__ size_t pool_block(const PoolView& v, int page, int h)
{
    return (static_cast<size_t>(page) * v.Hkv + h) * pool_block_bytes<D, INT4>(v);
}

// Page of token j of sequence b, or -1 where the table or the pool has none.
__device__ __forceinline__ int pool_page(const PoolView& v, int b, long long j)
{
    if (j < 0 || (j >> v.page_shift) >= v.max_pages) return -1;
    const int page = v.table[static_cast<size_t>(b) * v.max_pages + (j >> v.page_shift)];
    return (page >= 0 && page < v.num_pages) ? page : -1;
}

// A block of packed rows t0 .. t0 + n - 1 finds each row's sequence: seq[i] (preset to
// -1, published by the caller's barrier) becomes the b with cu[b] <= t0 + i < cu[b + 1].
__device__ __forceinline__ void find_sequences(const int* cu, int B, int t0, int n, int* seq)
{
    for (int b = threadIdx.x; b < B; b += blockDim.x) {
        const int lo = max(cu[b], t0), hi = min(cu[b + 1], t0 + n);
        for (int t = lo; t < hi; ++t) seq[t - t0] = b;
    }
}

// ---------------------------------------------------------------------------------
// Append.  Bound by memory: q, k and v are read once and written once.  A block takes
// `tpb` consecutive tokens with all their heads, so that the sines and cosines of a
// token are computed once and shared by its heads through shared memory.
//
// Angles: with F = inv_freq / (2 pi) as a fraction of a turn in 64-bit fixed point,
// position * F modulo 2^64 is the angle in turns reduced exactly (the wrap-around of the
// integer product drops whole turns), whatever the position; the error is inv_freq's
// rounding to 2^-53 relative, times the position.
//
// A row is cut into items of two 16-byte vectors that hold both members of their pairs
// (half-split pairs: vectors i and i + rot / 16; interleaved or not rotated: two
// neighbours), so that a thread can overwrite what it read (q_out = q).
// ---------------------------------------------------------------------------------
struct AppendParams {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride;
    void* q_out;
    void *k_cache, *v_cache;
    const int *cu, *seqlens_k;
    const float* inv_freq;
    PoolView pool;
    int rot, interleaved, B, total, Hq, tpb;
};

constexpr int kAppendTokens = 4;  // most tokens of a block

struct AppendToken {
    int seq, pos, page, slot;
};

// Vectors (first, second) of item i of a row, and whether it is rotated.
template <int D>
__device__ __forceinline__ bool append_item(int i, int rot, bool interleaved, int& a, int& b)
{
    const int rv = rot / 16;
    const bool turned = i < rv;
    if (turned && !interleaved) {
        a = i;
        b = i + rv;
    } else {
        a = 2 * i;
        b = a + 1;
    }
    return turned;
}

// Turns the 16 values of an item; angle r of the item at cs[r * pitch].
__device__ __forceinline__ void turn_item(float (&x)[8], float (&y)[8], const float2* cs, int pitch, bool interleaved)
{
    if (!interleaved) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const float2 c = cs[r * pitch];
            const float u = x[r], w = y[r];
            x[r] = u * c.x - w * c.y;
            y[r] = w * c.x + u * c.y;
        }
    } else {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const float2 c = cs[r * pitch];
            float* z = r < 4 ? x : y;
            const float u = z[2 * (r & 3)], w = z[2 * (r & 3) + 1];
            z[2 * (r & 3)] = u * c.x - w * c.y;
            z[2 * (r & 3) + 1] = w * c.x + u * c.y;
        }
    }
}

// Eight codes of a group of 32 spread over four neighbouring lanes, x in 64 bits: the
// codes' borders are decided exactly, so that the pool's contents do not depend on the
// order of a sum.  Returns the codes (four bits each, x[0] lowest) and the pair word.
template <bool BF16>
__device__ __forceinline__ uint32_t quantise8(const double (&x)[8], uint32_t& pair)
{
    double lo = x[0], hi = x[0];
    int bad = !isfinite(x[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        lo = fmin(lo, x[i]);
        hi = fmax(hi, x[i]);
        bad |= !isfinite(x[i]);
    }
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        lo = fmin(lo, __shfl_xor_sync(0xffffffffu, lo, m));
        hi = fmax(hi, __shfl_xor_sync(0xffffffffu, hi, m));
        bad |= __shfl_xor_sync(0xffffffffu, bad, m);
    }
    const double zero = pg_unpack2<BF16>(pg_pack2<BF16>(static_cast<float>(lo), 0.0f)).x;
    const float range = static_cast<float>(fmax(hi - zero, 0.0) / 15.0);
    pair = pg_pack2<BF16>(range, static_cast<float>(zero));
    const double scale = pg_unpack2<BF16>(pair).x;
    if (bad || !isfinite(zero) || !isfinite(scale)) {
        pair = 0x7fff7fffu;  // a NaN in both types
        return 0u;
    }
    if (!(scale > 0.0)) return 0u;
    const double inv = 1.0 / scale;
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const double d = x[i] - zero;
        double c = rint(d * inv);
        // next to a border the quotient itself decides (the product may be an ulp off)
        if (fabs(d * inv - c) > 0.499999) c = rint(d / scale);
        codes |= static_cast<uint32_t>(static_cast<int>(fmin(fmax(c, 0.0), 15.0))) << (4 * i);
    }
    return codes;
}

template <int D, bool BF16, bool INT4>
__global__ void __launch_bounds__(256) fa_kv_append_kernel(const AppendParams p)
{
    constexpr int VPR = D / 8;  // 16-byte vectors per row
    constexpr int IPR = D / 16; // items per row
    __shared__ AppendToken tok[kAppendTokens];
    __shared__ int seq[kAppendTokens];
    // angle a of token i: plane a % 8, column a / 8 (an item's eight angles are eight planes)
    __shared__ float2 cs[kAppendTokens][8][IPR];
    __shared__ double2 csd[INT4 ? kAppendTokens : 1][8][INT4 ? IPR : 1];
    const int t0 = blockIdx.x * p.tpb;
    const int n = min(p.tpb, p.total - t0);
    const int tid = threadIdx.x;
    const bool interleaved = p.interleaved != 0;

    if (tid < n) seq[tid] = -1;
    __syncthreads();
    find_sequences(p.cu, p.B, t0, n, seq);
    __syncthreads();
    if (tid < n) {
        AppendToken k{seq[tid], 0, -1, 0};
        if (k.seq >= 0) {
            const long long pos = static_cast<long long>(p.seqlens_k[k.seq]) - p.cu[k.seq + 1] + (t0 + tid);
            k.pos = static_cast<int>(pos);
            k.page = pool_page(p.pool, k.seq, pos);
            k.slot = k.pos & (p.pool.page_size - 1);
            if (k.page < 0) record_bad_page(PAGED_APPEND);
        }
        tok[tid] = k;
    }
    __syncthreads();
    const int half = p.rot / 2;
    for (int e = tid; e < n * half; e += blockDim.x) {
        const int i = e / half, a = e - i * half;
        double f = static_cast<double>(p.inv_freq[a]) * 0.15915494309189535;  // turns per position
        f -= rint(f);
        const unsigned long long step = 2ull * static_cast<unsigned long long>(__double2ll_rn(f * 9223372036854775808.0));
        const long long turn = static_cast<long long>(step * static_cast<unsigned long long>(static_cast<long long>(tok[i].pos)));
        if constexpr (INT4) {
            double s, c;
            sincospi(static_cast<double>(turn) * (1.0 / 9223372036854775808.0), &s, &c);
            csd[i][a & 7][a >> 3] = make_double2(c, s);
            cs[i][a & 7][a >> 3] = make_float2(static_cast<float>(c), static_cast<float>(s));
        } else {
            float s, c;
            sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * (1.0f / 2147483648.0f), &s, &c);
            cs[i][a & 7][a >> 3] = make_float2(c, s);
        }
    }
    __syncthreads();

    // queries, and with 16-bit pages keys and values
    const int qi = p.q != nullptr ? p.Hq * IPR : 0;
    const int ki = INT4 ? 0 : p.pool.Hkv * IPR;
    const int per = qi + 2 * ki;
    for (int e = tid; e < n * per; e += blockDim.x) {
        const int i = e / per;
        int r = e - i * per;
        const AppendToken k = tok[i];
        if (k.seq < 0) continue;
        const int t = t0 + i;
        const uint16_t* src;
        uint16_t* dst;
        bool may_turn = true;
        int h;
        if (r < qi) {
            h = r / IPR;
            r -= h * IPR;
            src = static_cast<const uint16_t*>(p.q) + t * p.q_stride + h * D;
            dst = static_cast<uint16_t*>(p.q_out) + (static_cast<size_t>(t) * p.Hq + h) * D;
        } else {
            if (k.page < 0) continue;
            r -= qi;
            may_turn = r < ki;
            if (!may_turn) r -= ki;
            h = r / IPR;
            r -= h * IPR;
            src = may_turn ? static_cast<const uint16_t*>(p.k) + t * p.k_stride + h * D
                           : static_cast<const uint16_t*>(p.v) + t * p.v_stride + h * D;
            dst = static_cast<uint16_t*>(may_turn ? p.k_cache : p.v_cache) +
                  pool_block<D, false>(p.pool, k.page, h) / 2 + static_cast<size_t>(k.slot) * D;
        }
        int a, b;
        const bool turned = append_item<D>(r, p.rot, interleaved, a, b) && may_turn;
        uint4 u = reinterpret_cast<const uint4*>(src)[a], w = reinterpret_cast<const uint4*>(src)[b];
        if (turned) {
            float x[8], y[8];
            pg_unpack8<BF16>(u, x);
            pg_unpack8<BF16>(w, y);
            turn_item(x, y, &cs[i][0][r], IPR, interleaved);
            u = pg_pack8<BF16>(x);
            w = pg_pack8<BF16>(y);
        }
        reinterpret_cast<uint4*>(dst)[a] = u;
        reinterpret_cast<uint4*>(dst)[b] = w;
    }

    if constexpr (INT4) {
        const int kv = p.pool.Hkv * VPR;
        const int count = n * 2 * kv;
        for (int e0 = tid & ~31; e0 < count; e0 += blockDim.x) {  // whole warps: lanes of a group exchange
            const int e = min(e0 + (tid & 31), count - 1);
            const int i = e / (2 * kv);
            int r = e - i * 2 * kv;
            const bool key = r < kv;
            if (!key) r -= kv;
            const int h = r / VPR, u = r - h * VPR;  // vector u of head h
            const AppendToken k = tok[i];
            const int t = t0 + i;
            double x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.0;
            if (k.page >= 0) {
                const uint4* src = reinterpret_cast<const uint4*>(
                    key ? static_cast<const uint16_t*>(p.k) + t * p.k_stride + h * D
                        : static_cast<const uint16_t*>(p.v) + t * p.v_stride + h * D);
                float f[8];
                pg_unpack8<BF16>(src[u], f);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = f[j];
                const int rv = p.rot / 16;
                if (key && u < 2 * rv) {
                    if (!interleaved) {
                        const bool low = u < rv;
                        const int c0 = low ? u : u - rv;
                        pg_unpack8<BF16>(src[low ? u + rv : c0], f);
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            const double2 c = csd[i][j][c0];
                            x[j] = low ? x[j] * c.x - f[j] * c.y : x[j] * c.x + f[j] * c.y;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const double2 c = csd[i][(4 * u + j) & 7][u >> 1];
                            const double a = x[2 * j], b = x[2 * j + 1];
                            x[2 * j] = a * c.x - b * c.y;
                            x[2 * j + 1] = b * c.x + a * c.y;
                        }
                    }
                }
            }
            uint32_t pair;
            const uint32_t codes = quantise8<BF16>(x, pair);
            if (e0 + (tid & 31) >= count || k.page < 0) continue;
            uint8_t* blk = static_cast<uint8_t*>(key ? p.k_cache : p.v_cache) + pool_block<D, true>(p.pool, k.page, h);
            reinterpret_cast<uint32_t*>(blk + static_cast<size_t>(k.slot) * (D / 2))[u] = codes;
            if ((u & 3) == 0)
                reinterpret_cast<uint32_t*>(blk + static_cast<size_t>(p.pool.page_size) * (D / 2) +
                                            static_cast<size_t>(k.slot) * (D / 8))[u >> 2] = pair;
        }
    }
}

// ---------------------------------------------------------------------------------
// Read-back.  Bound by memory.  A block takes kGatherTokens consecutive packed rows;
// thread = one 16-byte vector of a row.
// ---------------------------------------------------------------------------------
struct GatherParams {
    const void *k_cache, *v_cache;
    void *k, *v;
    const int* cu;
    PoolView pool;
    int B, total;
};

constexpr int kGatherTokens = 16;

// Eight values (vector u) of a 4-bit row.
template <int D, bool BF16>
__device__ __forceinline__ void read_codes(const uint8_t* blk, const PoolView& v, int slot, int u, float (&x)[8])
{
    const uint32_t c = reinterpret_cast<const uint32_t*>(blk + static_cast<size_t>(slot) * (D / 2))[u];
    const float2 sz = pg_unpack2<BF16>(reinterpret_cast<const uint32_t*>(
        blk + static_cast<size_t>(v.page_size) * (D / 2) + static_cast<size_t>(slot) * (D / 8))[u >> 2]);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = fmaf(static_cast<float>((c >> (4 * j)) & 15u), sz.x, sz.y);
}

template <int D, bool BF16, bool INT4>
__device__ __forceinline__ uint4 read_vector(const uint8_t* blk, const PoolView& v, int slot, int u)
{
    if constexpr (!INT4) {
        return reinterpret_cast<const uint4*>(blk + static_cast<size_t>(slot) * (2 * D))[u];
    } else {
        float x[8];
        read_codes<D, BF16>(blk, v, slot, u, x);
        return pg_pack8<BF16>(x);
    }
}

template <int D, bool BF16, bool INT4>
__global__ void __launch_bounds__(256) fa_kv_gather_kernel(const GatherParams p)
{
    constexpr int VPR = D / 8;
    __shared__ int seq[kGatherTokens], page[kGatherTokens], slot[kGatherTokens];
    const int t0 = blockIdx.x * kGatherTokens;
    const int n = min(kGatherTokens, p.total - t0);
    const int tid = threadIdx.x;
    if (tid < n) seq[tid] = -1;
    __syncthreads();
    find_sequences(p.cu, p.B, t0, n, seq);
    __syncthreads();
    if (tid < n && seq[tid] >= 0) {
        const int j = t0 + tid - p.cu[seq[tid]];
        page[tid] = pool_page(p.pool, seq[tid], j);
        slot[tid] = j & (p.pool.page_size - 1);
        if (page[tid] < 0) record_bad_page(PAGED_GATHER);
    }
    __syncthreads();
    const int row = p.pool.Hkv * VPR;
    for (int e = tid; e < n * 2 * row; e += blockDim.x) {
        const int i = e / (2 * row);
        if (seq[i] < 0) continue;
        int r = e - i * 2 * row;
        const bool key = r < row;
        if (!key) r -= row;
        const int h = r / VPR, u = r - h * VPR;
        uint4 x = make_uint4(0u, 0u, 0u, 0u);
        if (page[i] >= 0)
            x = read_vector<D, BF16, INT4>(static_cast<const uint8_t*>(key ? p.k_cache : p.v_cache) +
                                               pool_block<D, INT4>(p.pool, page[i], h),
                                           p.pool, slot[i], u);
        reinterpret_cast<uint4*>(static_cast<uint16_t*>(key ? p.k : p.v) +
                                 (static_cast<size_t>(t0 + i) * p.pool.Hkv + h) * D)[u] = x;
    }
}

}  // namespace fa
