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
// Measured (time on the GPU): 12,313 tokens, 32/8 heads of 128, 16-bit pages: 52 us, 5.9
// TB/s; 15,530 tokens, 32/4 heads, 4-bit pages: 73 us, 1.6 times its bytes (keys are
// turned and coded in 64 bits; 60 % of the issue slots and 43 % of the ALU pipe are used);
// 32 tokens: 4.2 us, the latency of three loads in turn.  Four tokens per block beat two
// (54 against 58 us) and eight (56).
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

// Eight codes of a group of 32 spread over four neighbouring lanes.  T is a type that
// holds the values exactly, or as exactly as 64 bits do (rotated keys): the group's zero
// and scale are formed in 64 bits, and so is a code whose value lies next to a border
// between two (one in some thousands); the other codes are told apart in 32 bits, whose
// quotient is off by less than 2^-18 (three roundings of at most 16).  Returns the codes
// (four bits each, x[0] lowest) and the pair word.
template <bool BF16, class T>
__device__ __forceinline__ uint32_t quantise8(const T (&x)[8], uint32_t& pair)
{
    T lo = x[0], hi = x[0];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = x[i] < lo ? x[i] : lo;
        hi = x[i] > hi ? x[i] : hi;
        bad |= !(x[i] - x[i] == T(0));  // an infinity or a NaN
    }
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        const T a = __shfl_xor_sync(0xffffffffu, lo, m), b = __shfl_xor_sync(0xffffffffu, hi, m);
        lo = a < lo ? a : lo;
        hi = b > hi ? b : hi;
    }
    const uint32_t votes = __ballot_sync(0xffffffffu, bad);
    bad = (votes >> (threadIdx.x & 28) & 15u) != 0u;
    const double zero = pg_unpack2<BF16>(pg_pack2<BF16>(static_cast<float>(lo), 0.0f)).x;
    const float range = static_cast<float>(fmax(static_cast<double>(hi) - zero, 0.0) / 15.0);
    pair = pg_pack2<BF16>(range, static_cast<float>(zero));
    const float scale = pg_unpack2<BF16>(pair).x;
    if (bad || !isfinite(zero) || !isfinite(scale)) {
        pair = 0x7fff7fffu;  // a NaN in both types
        return 0u;
    }
    if (!(scale > 0.0f)) return 0u;
    // Powers of two keep the quotient's terms inside the 32-bit range for any scale.  Where
    // scales are large so may the values be, and a difference of two reaches twice the range
    // (turned keys: 2.5 times): a sixteenth of it is formed, by one multiply-add
    const T part = scale < 1.0f ? T(1) : T(0.0625), low = static_cast<T>(zero) * part;
    const float up = scale < 1.0f ? 0x1p100f : 0x1p-96f;
    const float inv = 1.0f / (scale * (scale < 1.0f ? 0x1p100f : 0x1p-100f));
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = static_cast<float>(fma(x[i], part, -low)) * up * inv;
        const float r = fminf(fmaxf(q, 0.0f), 15.0f);
        const float t = r + 12582912.0f;  // 1.5 * 2^23: rounds to a whole number
        uint32_t c = __float_as_uint(t) & 15u;
        if (fabsf(r - (t - 12582912.0f)) > 0.4999f) {
            const double e = rint((static_cast<double>(x[i]) - zero) / static_cast<double>(scale));
            c = static_cast<uint32_t>(static_cast<int>(fmin(fmax(e, 0.0), 15.0)));
        }
        codes |= c << (4 * i);
    }
    return codes;
}

template <int D, bool BF16, bool INT4>
__global__ void __launch_bounds__(256, 4) fa_kv_append_kernel(const AppendParams p)
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

    // queries, and with 16-bit pages keys and values: a thread's item of every token
    const int qi = p.q != nullptr ? p.Hq * IPR : 0;
    const int ki = INT4 ? 0 : p.pool.Hkv * IPR;
    for (int e = tid; e < qi + 2 * ki; e += blockDim.x) {
        const bool query = e < qi;
        const bool key = !query && e < qi + ki;
        int r = query ? e : key ? e - qi : e - qi - ki;
        const int h = r / IPR;
        r -= h * IPR;
        int a, b;
        const bool turned = append_item<D>(r, p.rot, interleaved, a, b) && (query || key);
        const uint16_t* src = static_cast<const uint16_t*>(query ? p.q : key ? p.k : p.v) + h * D;
        const long long stride = query ? p.q_stride : key ? p.k_stride : p.v_stride;
        uint4 u[kAppendTokens], w[kAppendTokens];
#pragma unroll
        for (int i = 0; i < kAppendTokens; ++i) {
            if (i >= n || tok[i].seq < 0) continue;
            const uint4* s = reinterpret_cast<const uint4*>(src + (t0 + i) * stride);
            u[i] = s[a];
            w[i] = s[b];
        }
#pragma unroll
        for (int i = 0; i < kAppendTokens; ++i) {
            if (i >= n || tok[i].seq < 0 || (!query && tok[i].page < 0)) continue;
            if (turned) {
                float x[8], y[8];
                pg_unpack8<BF16>(u[i], x);
                pg_unpack8<BF16>(w[i], y);
                turn_item(x, y, &cs[i][0][r], IPR, interleaved);
                u[i] = pg_pack8<BF16>(x);
                w[i] = pg_pack8<BF16>(y);
            }
            uint4* dst;
            if (query)
                dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q_out) + (static_cast<size_t>(t0 + i) * p.Hq + h) * D);
            else
                dst = reinterpret_cast<uint4*>(static_cast<uint8_t*>(key ? p.k_cache : p.v_cache) +
                                               pool_block<D, false>(p.pool, tok[i].page, h) +
                                               static_cast<size_t>(tok[i].slot) * (2 * D));
            dst[a] = u[i];
            dst[b] = w[i];
        }
    }

    if constexpr (INT4) {
        // a vector at a time; whole warps, since the lanes of a group exchange
        const int kv = p.pool.Hkv * VPR;
        const int rv = p.rot / 16;
        const int count = n * 2 * kv;
        for (int e0 = tid & ~31; e0 < count; e0 += blockDim.x) {
            int e = min(e0 + (tid & 31), count - 1);
            const int i = e / (2 * kv);
            e -= i * 2 * kv;
            const bool key = e < kv;
            const int h = (key ? e : e - kv) / VPR, u = (key ? e : e - kv) - h * VPR;  // vector u of head h
            const bool turned = key && u < 2 * rv;
            const bool mine = e0 + (tid & 31) < count && tok[i].page >= 0;
            // the vector with the other members of its pairs
            const int other = !turned || interleaved ? u : u < rv ? u + rv : u - rv;
            uint4 in = make_uint4(0u, 0u, 0u, 0u), part = in;
            if (mine) {
                const uint4* const row = reinterpret_cast<const uint4*>(
                    static_cast<const uint16_t*>(key ? p.k : p.v) + (t0 + i) * (key ? p.k_stride : p.v_stride) + h * D);
                in = row[u];
                part = row[other];
            }
            float f[8];
            pg_unpack8<BF16>(in, f);
            uint32_t pair, codes;
            if (__any_sync(0xffffffffu, turned)) {
                double x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = f[j];
                if (turned && !interleaved) {
                    const bool low = u < rv;
                    pg_unpack8<BF16>(part, f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const double2 c = csd[i][j][low ? u : other];
                        x[j] = low ? x[j] * c.x - f[j] * c.y : x[j] * c.x + f[j] * c.y;
                    }
                } else if (turned) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const double2 c = csd[i][(4 * u + j) & 7][u >> 1];
                        const double a = x[2 * j], b = x[2 * j + 1];
                        x[2 * j] = a * c.x - b * c.y;
                        x[2 * j + 1] = b * c.x + a * c.y;
                    }
                }
                codes = quantise8<BF16>(x, pair);
            } else {
                codes = quantise8<BF16>(f, pair);
            }
            if (!mine) continue;
            uint8_t* blk = static_cast<uint8_t*>(key ? p.k_cache : p.v_cache) + pool_block<D, true>(p.pool, tok[i].page, h);
            reinterpret_cast<uint32_t*>(blk + static_cast<size_t>(tok[i].slot) * (D / 2))[u] = codes;
            if ((u & 3) == 0)
                reinterpret_cast<uint32_t*>(blk + static_cast<size_t>(p.pool.page_size) * (D / 2) +
                                            static_cast<size_t>(tok[i].slot) * (D / 8))[u >> 2] = pair;
        }
    }
}

// ---------------------------------------------------------------------------------
// Expanding codes, two at a time.
// ---------------------------------------------------------------------------------
template <bool BF16>
__device__ __forceinline__ uint32_t fma16x2(uint32_t a, uint32_t b, uint32_t c)
{
    uint32_t d;
    if constexpr (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

template <bool BF16>
__device__ __forceinline__ uint32_t add16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    if constexpr (BF16) asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Codes in a 32-bit word, in bits 0 .. 3 (HIGH: 4 .. 7) of both halves.
template <bool HIGH>
__device__ __forceinline__ uint32_t code_tiny(uint32_t w)
{
    return w & (HIGH ? 0x00f000f0u : 0x000f000fu);
}
// scale * code + zero of a pair.  s4: 4 scale (bf16).
template <bool BF16, bool HIGH>
__device__ __forceinline__ uint32_t code_value(uint32_t w, uint32_t s, uint32_t s4, uint32_t z)
{
    if constexpr (BF16 && HIGH)  // 2^-129 code, times 2^127
        return fma16x2<true>(mul_bf16x2(w & 0x00f000f0u, 0x7f007f00u), s4, z);
    else if constexpr (BF16)     // 128 + code
        return fma16x2<true>(add16x2<true>((w & 0x000f000fu) | 0x43004300u, 0xc300c300u), s, z);
    else if constexpr (HIGH)     // 64 + code
        return fma16x2<false>(add16x2<false>((w & 0x00f000f0u) | 0x54005400u, 0xd400d400u), s, z);
    else                         // 1024 + code
        return fma16x2<false>(add16x2<false>((w & 0x000f000fu) | 0x64006400u, 0xe400e400u), s, z);
}

// ---------------------------------------------------------------------------------
// Read-back.  Bound by memory.  A block takes kGatherTokens consecutive packed rows; a
// thread takes one 16-byte vector (head, place) of every row, so that its addresses
// differ from row to row by the row's place in the pool alone.
// ---------------------------------------------------------------------------------
struct GatherParams {
    const void *k_cache, *v_cache;
    void *k, *v;
    const int* cu;
    PoolView pool;
    int B, total;
};

constexpr int kGatherTokens = 16;

// Vector u of a row: scale * code + zero with one rounding.
template <int D, bool BF16, bool INT4>
__device__ __forceinline__ uint4 read_vector(const uint8_t* row, const uint8_t* pairs, int u)
{
    if constexpr (!INT4) {
        return reinterpret_cast<const uint4*>(row)[u];
    } else {
        const uint32_t w = reinterpret_cast<const uint32_t*>(row)[u];
        const uint32_t sz = reinterpret_cast<const uint32_t*>(pairs)[u >> 2];
        const uint32_t s = __byte_perm(sz, sz, 0x1010), z = __byte_perm(sz, sz, 0x3232);
        const uint32_t s4 = BF16 ? mul_bf16x2(s, 0x40804080u) : s;
        // pairs (i, i + 4)
        const uint32_t a = code_value<BF16, false>(w, s, s4, z), b = code_value<BF16, true>(w, s, s4, z);
        const uint32_t c = code_value<BF16, false>(w >> 8, s, s4, z), d = code_value<BF16, true>(w >> 8, s, s4, z);
        return make_uint4(__byte_perm(a, b, 0x5410), __byte_perm(c, d, 0x5410), __byte_perm(a, b, 0x7632),
                          __byte_perm(c, d, 0x7632));
    }
}

template <int D, bool BF16, bool INT4>
__global__ void __launch_bounds__(256, INT4 ? 6 : 4) fa_kv_gather_kernel(const GatherParams p)
{
    constexpr int VPR = D / 8;
    constexpr int RB = INT4 ? D / 2 : 2 * D;
    __shared__ int seq[kGatherTokens];
    // offset of the row in head 0 of its page (-1: no page; -2: no sequence), and its slot
    __shared__ long long off[kGatherTokens];
    __shared__ int slot[kGatherTokens];
    const int t0 = blockIdx.x * kGatherTokens;
    const int n = min(kGatherTokens, p.total - t0);
    const int tid = threadIdx.x;
    if (tid < n) seq[tid] = -1;
    __syncthreads();
    find_sequences(p.cu, p.B, t0, n, seq);
    __syncthreads();
    if (tid < kGatherTokens) {
        long long o = -2;
        if (tid < n && seq[tid] >= 0) {
            const int j = t0 + tid - p.cu[seq[tid]];
            const int page = pool_page(p.pool, seq[tid], j);
            slot[tid] = j & (p.pool.page_size - 1);
            o = page < 0 ? -1 : static_cast<long long>(pool_block<D, INT4>(p.pool, page, 0)) + slot[tid] * RB;
            if (page < 0) record_bad_page(PAGED_GATHER);
        }
        off[tid] = o;
    }
    __syncthreads();
    const int row = p.pool.Hkv * VPR;
    for (int e = tid; e < 2 * row; e += blockDim.x) {
        const bool key = e < row;
        const int r = key ? e : e - row;
        const int h = r / VPR, u = r - h * VPR;
        const uint8_t* const src = static_cast<const uint8_t*>(key ? p.k_cache : p.v_cache) +
                                   static_cast<size_t>(h) * pool_block_bytes<D, INT4>(p.pool);
        uint4* const dst = static_cast<uint4*>(key ? p.k : p.v) + static_cast<size_t>(t0) * row + r;
        // rows whose loads are in flight together.  4-bit pools: writing is three quarters of the
        // traffic, and one row after the other leaves in order (142 us against 162 with two
        // and 187 with eight, 134,452 tokens of 8 heads of 128); 16-bit: eight (37.5 us
        // against 47 with one, 49,675 tokens of 2 heads of 256)
        constexpr int AT_ONCE = INT4 ? 1 : 8;
#pragma unroll 1
        for (int i0 = 0; i0 < kGatherTokens; i0 += AT_ONCE) {
            uint4 x[AT_ONCE];
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i) {
                x[i] = make_uint4(0u, 0u, 0u, 0u);
                const long long o = off[i0 + i];
                if (o >= 0) {
                    const uint8_t* const at = src + o;
                    x[i] = read_vector<D, BF16, INT4>(at, at + p.pool.page_size * RB - slot[i0 + i] * (RB - D / 8), u);
                }
            }
#pragma unroll
            for (int i = 0; i < AT_ONCE; ++i)
                if (off[i0 + i] != -2) dst[static_cast<size_t>(i0 + i) * row] = x[i];
        }
    }
}

}  // namespace fa
