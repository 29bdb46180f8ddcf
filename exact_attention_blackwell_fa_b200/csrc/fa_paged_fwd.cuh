// fa_paged_fwd.cuh -- attention over the paged cache, for few query rows per sequence.
//
//   O = softmax(scale Q K^T [+ causal]) V, LSE, K and V read from the pools.
//
// Bound by memory: every cached token is read once for all the query heads that share
// its KV head, and a decode step does only 2 * group products per cached value.  So:
//
//   * a work unit is (sequence, block of 8 NT query rows, KV head), its rows being
//     (query, head of the group) pairs; a unit's keys are cut into granules of W * TS
//     tokens, and the granules of all units, in order, into as many equal ranges as
//     there are resident CTAs -- whatever the lengths, every CTA streams the same
//     number of tokens.  Lengths are read on the device.  A unit that falls into one
//     range is written directly; the pieces of one that was cut go to the workspace in
//     fp32 and a second, small launch joins them in a fixed order;
//   * each warp streams its own TS tokens of a granule through its own ring of
//     shared-memory slots with cp.async (rows past the end or without a page are filled
//     with zeros, so nothing a pool holds there can reach a sum) and keeps its own
//     running maximum, sum and O; the warps of a CTA meet only at the end of a unit.
//     The ring runs ahead across units;
//   * scores are computed transposed, S^T = K Q^T with the tokens as the 16 rows of an
//     mma tile and the query rows as its 8 columns, so that one to eight heads of a
//     group cost one tile; O^T = V^T P^T likewise.  Tensor time is far below the
//     memory time at these row counts, which is why the warp-level mma is used: its
//     operands are registers, where the 4-bit codes are expanded;
//   * P is split into two 16-bit terms (two products), so that its rounding does not
//     add to the output's own: a weight is held to 2^-16 of itself in bf16, and in fp16
//     to 2^-20 of itself or 2^-25, half the type's least step.  For that fp16 weights
//     are taken 2^14 times larger: half the least step is then 2^-39 of a row's largest
//     weight at most, and a token 18 nats below the largest is still held to 2^-13.
//
// 4-bit keys: the four bits of a code, masked in place out of a 32-bit word, are a
// 16-bit float far below 1 whose value is code * 2^-133 (bf16) or code * 2^-24 (fp16),
// 16 times that for the second code of a byte (exponents 0 and 1 have the same step, so
// the pattern is linear in the code).  One instruction therefore expands two codes.  The
// query rows are scaled by a power of two so that the products stay in range (those of
// the 16 times larger codes by 2^-4 of that), and each group's product is multiplied by
// the token's scale in fp32; zero * (sum of the query over the group) is added in fp32.
//
// 4-bit values: a code becomes a whole number of the type exactly (its bits under the
// exponent whose step is 1, that power of two taken off; or the tiny float multiplied
// up), and one fused multiply-add gives scale * code + zero with one rounding: the value
// that the read-back gives.
//
// Measured (time on the GPU; one B200, copy rate 6548 GB/s): 16-bit, 64 sequences up to
// 8192 tokens, 32/4 heads of 128: 91 us, 5.9 TB/s of keys and values, bound by memory (8
// us of it the prologue and the join); 4 x 131,072 tokens, 16/2 heads of 256: 164 us, 6.5
// TB/s.  4-bit, 64 sequences, 32/8 heads of 128: 103 us, 2.9 TB/s, where streaming alone
// takes 57 us: about 1000 instructions per 32 tokens of keys and values (22 % of them
// copies, addresses and page lookups), 58 % of the issue slots and 44 % of the ALU pipe
// used.  No unit is full: a warp's step is a chain (copy, scores, shuffles, exponentials,
// values) that 12 warps per SM do not cover.
#pragma once

#include <cfloat>
#include <utility>

#include "fa_paged.cuh"

namespace fa {

// ---------------------------------------------------------------------------------
// Warp-level products and copies
// ---------------------------------------------------------------------------------
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8).  Lane 4 g + t: A rows g, g + 8, columns
// 2 t, 2 t + 1 (and + 8); B column g, rows 2 t, 2 t + 1 (and + 8); D rows g, g + 8,
// columns 2 t, 2 t + 1.
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// D = A B
template <bool BF16>
__device__ __forceinline__ void mma16816_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
// Transpose of an 8 x 8 matrix of 16-bit values (lane 4 g + t: row g, columns 2 t, 2 t + 1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// 16 bytes global -> shared, both at constant offsets; of the second form only the first
// `bytes` (0 .. 16) are read, the rest is zero.
template <int TO, int FROM>
__device__ __forceinline__ void copy16(uint32_t dst, const void* src)
{
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
                 "n"(TO), "n"(FROM)
                 : "memory");
}
__device__ __forceinline__ void copy16_part(uint32_t dst, const void* src, uint32_t bytes)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <class T>
__device__ __forceinline__ T lds(const uint8_t* a)
{
    return *reinterpret_cast<const T*>(a);
}
// ---------------------------------------------------------------------------------
// Parameters
// ---------------------------------------------------------------------------------
// Division of 0 .. 2^31 - 1 by a number that a launch knows: with 2^(s-1) < d <= 2^s and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (n + (n m >> 32)) >> s.
struct Divider {
    uint32_t d, m, s;
    __host__ static Divider by(uint32_t d)
    {
        uint32_t s = 0;
        while ((1ull << s) < d) ++s;
        return {d, static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1), s};
    }
    __device__ __forceinline__ int quotient(int n) const
    {
        return static_cast<int>((__umulhi(static_cast<uint32_t>(n), m) + static_cast<uint32_t>(n)) >> s);
    }
    __device__ __forceinline__ int remainder(int n) const { return n - quotient(n) * static_cast<int>(d); }
};

// A unit that was cut: its pieces are slot 2 i + 1 of the CTA i that writes the record
// and slots 2 j of the CTAs i < j <= last (a sum of 0 where a range was empty).
struct PagedRecord {
    int b, u, last;  // last < 0: nothing to join
    int pad;
};

struct PagedFwdParams {
    const void* q;
    const void *k_cache, *v_cache;
    void* o;
    float* lse;
    const int *cu_q, *seqlens_k;
    PoolView pool;
    int B, max_q, total_q, Hq, group, causal;
    Divider by_group, by_hkv;
    float sl2;         // scale * log2(e)
    uint32_t block_bytes;  // of a (page, head)
    int coarse;        // granules that ranges keep together
    float* opart;      // [2 grid][rows of a unit][D]
    float2* mlpart;    // [2 grid][rows of a unit] (reference maximum, sum)
    PagedRecord* rec;  // [grid]
};

// CTAs per SM, at most; the workspace has pieces for as many.
constexpr int kPagedCtas = 2;

template <int D, bool INT4, int NT>
struct PagedCfg {
    // Tokens of a warp's step, and warps of a CTA.  Rows of d = 128 for one tile: six warps
    // of 168 registers, two CTAs per SM (64 sequences up to 8192 tokens: 16-bit 96.0 us
    // against 98.7 with four and 98.4 with eight; 4-bit 105 us against 120 with five, 127
    // and 123 with seven and eight, which spill).  4-bit rows of 384 and 512 fill the shared
    // memory with few slots: halving the step makes room for twice the warps (d = 512, 32
    // sequences of 8192 tokens: 82 us against 106).  Two and four tiles take four warps,
    // whose 255 registers they need; other counts were not measured for them
    static constexpr int TS = INT4 && D < 384 ? 32 : 16;
    static constexpr int MB = TS / 16;
    static constexpr int W = INT4 && D >= 384 ? 8 : D == 128 && NT == 1 ? 6 : 4;
    static constexpr int ROWS = 8 * NT;
    static constexpr int GR = W * TS;              // tokens of a granule
    static constexpr int RB = INT4 ? D / 2 : 2 * D;  // bytes of a row (codes)
    static constexpr int RBS = RB <= 64 ? 64 : (RB + 127) / 128 * 128;  // its pitch
    static constexpr int SCB = INT4 ? D / 8 : 0;   // bytes of a row's (scale, zero) pairs
    static constexpr uint32_t SLOT = TS * (RBS + SCB);
    static constexpr int CTAS = D >= (INT4 ? 384 : 256) ? 1 : 2;
    static_assert(CTAS <= kPagedCtas, "workspace pieces");
    // Q of a unit, twice: the next unit's is fetched while the last one's O is joined.
    // B fragments [NT][D / 32][32 lanes][4], sums over groups [NT][D / 32][8], score
    // factors [NT][8]
    static constexpr uint32_t OFF_QS = NT * D * 16;
    static constexpr uint32_t OFF_F = OFF_QS + (INT4 ? NT * D : 0);
    static constexpr uint32_t Q_BYTES = OFF_F + NT * 32;
    static constexpr int DP = D <= 192 ? D : 128;  // dims of O joined at a time
    static constexpr int MP = DP + 4;              // their pitch, 4 mod 16: conflict-free
    static constexpr uint32_t OFF_Q = 0;
    static constexpr uint32_t OFF_ML = 2 * Q_BYTES;                    // [2][W][ROWS] (m, l)
    static constexpr uint32_t OFF_RED = OFF_ML + 2 * W * ROWS * 8;     // [W][8][MP]
    static constexpr uint32_t OFF_OK = OFF_RED + W * 8 * MP * 4;       // [W][8] blocks of a slot that have a page
    static constexpr uint32_t OFF_RING = (OFF_OK + W * 32 + 127u) & ~127u;
    // the rest are the warps' rings, K and V taking turns in their slots
    static constexpr uint32_t LIMIT = (CTAS == 1 ? 226 : 112) * 1024;
    static constexpr int NST_ = (LIMIT - OFF_RING) / (W * SLOT);
    // deeper rings of 16-bit rows are slower (d = 256, 4 sequences of 131,072 tokens: 168 us
    // with four slots, 183 with six): 64 to 128 KB in flight per SM cover the latency
    static constexpr int MOST = INT4 ? 6 : 4;
    static constexpr int NST = NST_ > MOST ? MOST : NST_;
    static_assert(NST >= 3, "ring depth");
    static constexpr uint32_t SMEM = OFF_RING + W * NST * SLOT;
    static constexpr int THREADS = W * 32;
    // 16-byte chunk c of row r lies at chunk c ^ key(r) of its 64- or 128-byte line, so
    // that the fragment loads of a warp meet no bank twice
    static constexpr int LINE = RBS == 64 ? 3 : 7;
    __device__ static constexpr int key(int r) { return RBS == 64 ? (r >> 1) & 3 : r & 7; }
};

// Lengths of sequence b as the kernels use them.
struct PagedSeq {
    int q0, Sq, Sk, nu;
    int kg, kt;  // granules of a unit, and pieces of `coarse` granules that ranges are cut from
};
template <class C>
__device__ __forceinline__ PagedSeq paged_seq(const PagedFwdParams& p, int b)
{
    PagedSeq s;
    s.q0 = p.cu_q[b];
    const long long end = p.cu_q[b + 1];
    s.Sq = s.q0 >= 0 && end <= p.total_q && end > s.q0 ? static_cast<int>(min(end - s.q0, static_cast<long long>(p.max_q))) : 0;
    s.Sk = max(0, min(p.seqlens_k[b], p.pool.max_pages << p.pool.page_shift));
    s.nu = static_cast<int>((static_cast<long long>(s.Sq) * p.group + C::ROWS - 1) / C::ROWS) * p.pool.Hkv;
    s.kg = s.Sk > 0 ? (s.Sk - 1) / C::GR + 1 : 1;
    s.kt = p.coarse > 1 ? (s.kg - 1) / p.coarse + 1 : s.kg;
    return s;
}

// Sum over the block (every thread gets it); `red` holds 33 values.
__device__ __forceinline__ long long block_sum(long long x, long long* red)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    long long s = 0;
    for (int i = 0; i < static_cast<int>(blockDim.x) / 32; ++i) s += red[i];
    return s;
}

// n / d, by 32 bits where they do
__device__ __forceinline__ long long divide(long long n, long long d)
{
    if (((n | d) >> 32) == 0) return static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
    return n / d;
}

// Where a CTA's range of granules begins: sequence b, granule `at` of its nu * kt.
struct PagedStart {
    int b;
    long long at, lo, hi, total;
};
template <class C>
__device__ __forceinline__ void paged_start(const PagedFwdParams& p, PagedStart* out, long long* red)
{
    const int T = blockDim.x, tid = threadIdx.x;
    auto granules = [&](int b) {
        if (b >= p.B) return 0ll;
        const PagedSeq s = paged_seq<C>(p, b);
        return static_cast<long long>(s.nu) * s.kt;
    };
    long long mine = granules(tid);
    const long long first = mine;
    for (int b = tid + T; b < p.B; b += T) mine += granules(b);
    if (blockIdx.x == 0)
        for (int b = tid; b < p.B; b += T)
            if (p.seqlens_k[b] > (p.pool.max_pages << p.pool.page_shift)) record_bad_page(PAGED_FWD);
    const long long total = block_sum(mine, red);
    const long long lo = divide(total * blockIdx.x, gridDim.x), hi = divide(total * (blockIdx.x + 1), gridDim.x);
    if (tid == 0) *out = PagedStart{0, 0, lo, hi, total};
    long long before = 0;
    for (int c = 0; c < p.B && before <= lo; c += T) {  // T sequences at a time: an inclusive sum over the block
        long long x = c == 0 ? first : granules(c + tid);
        const long long own = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if ((tid & 31) >= o) x += y;
        }
        __syncthreads();
        if ((tid & 31) == 31) red[tid >> 5] = x;
        __syncthreads();
        long long sum = 0;
        for (int i = 0; i < T / 32; ++i) {
            if (i < tid / 32) x += red[i];
            sum += red[i];
        }
        x += before;
        if (lo < hi && x - own <= lo && lo < x) {
            out->b = c + tid;
            out->at = lo - (x - own);
        }
        before += sum;
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------------
// A range's segments: parts of units, in order.
// ---------------------------------------------------------------------------------
struct PagedSegment {
    PagedSeq s;
    int b, u, g0, g1;
    int first, last;  // whether it begins and ends its unit
    int left;         // the unit's pieces past it
    int r0, R;     // first row of the unit, rows of the sequence
    int kmax;      // keys that some row of the unit sees
};
template <class C>
struct PagedWalk {
    PagedSeq s;
    int b, u, g;
    long long left;

    __device__ void init(const PagedFwdParams& p, const PagedStart& st)
    {
        b = st.b;
        left = st.hi - st.lo;
        if (left <= 0) return;
        s = paged_seq<C>(p, b);
        u = static_cast<int>(divide(st.at, s.kt));
        g = static_cast<int>(st.at - static_cast<long long>(u) * s.kt);
    }
    __device__ bool next(const PagedFwdParams& p, PagedSegment& x)
    {
        if (left <= 0) return false;
        while (u >= s.nu) {  // units are left, so a later sequence has them
            if (++b >= p.B) return false;
            u = 0;
            s = paged_seq<C>(p, b);
        }
        x.s = s;
        x.b = b;
        x.u = u;
        const int end = static_cast<int>(min(static_cast<long long>(s.kt), g + left));
        x.g0 = g * p.coarse;
        x.g1 = min(s.kg, end * p.coarse);
        x.first = g == 0;
        x.last = end == s.kt;
        x.left = s.kt - end;
        x.r0 = p.by_hkv.quotient(u) * C::ROWS;
        x.R = s.Sq * p.group;
        x.kmax = s.Sk;
        if (p.causal) {
            const int last = p.by_group.quotient(min(x.r0 + C::ROWS, x.R) - 1);
            x.kmax = max(0, min(s.Sk, last + s.Sk - s.Sq + 1));
        }
        left -= end - g;
        g = end;
        if (g == s.kt) {
            g = 0;
            ++u;
        }
        return true;
    }
};

// The steps of one warp, ahead of their use: the copies.  K and V take turns in the ring.
template <int D, bool INT4, int NT>
struct PagedLoad {
    using C = PagedCfg<D, INT4, NT>;
    PagedWalk<C> walk;
    PagedSegment seg;
    const int* table;    // the segment's pages
    int g, h;            // next granule and KV head of the segment
    bool more;
    // the step whose copies come next, and the one after it (its pages on their way):
    // its first token, keys that count, KV head, page of the lane's block of 16 tokens
    int base[2], kmax[2], hkv[2], page[2];
    long long off[C::MB];  // of the next step's blocks in the pools: their rows,
    int poff[C::MB];       // and from there their pairs
    uint32_t bits;         // which of them have a page
    uint32_t slot, ok;     // shared-memory addresses of this warp's next slot and its page bits
    uint32_t n = 0;        // slot

    __device__ void init(const PagedFwdParams& p, const PagedStart& st, uint32_t ring_, uint32_t ok_)
    {
        slot = ring_;
        ok = ok_;
        walk.init(p, st);
        segment(p);
        fetch(p, 0);
        fetch(p, 1);
    }
    __device__ void segment(const PagedFwdParams& p)
    {
        more = walk.next(p, seg);
        if (!more) return;
        g = seg.g0;
        h = p.by_hkv.remainder(seg.u);
        table = p.pool.table + static_cast<size_t>(seg.b) * p.pool.max_pages;
    }
    // the warp's next step into entry i; base < 0: none is left
    __device__ void fetch(const PagedFwdParams& p, int i)
    {
        const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
        base[i] = -1;
        while (more) {
            // granules start below 2^31, their last tokens need not
            const uint32_t at = static_cast<uint32_t>(g) * C::GR + w * C::TS;
            if (g < seg.g1 && at < static_cast<uint32_t>(seg.kmax)) {
                ++g;
                base[i] = static_cast<int>(at);
                kmax[i] = seg.kmax;
                hkv[i] = h;
                const int j = static_cast<int>(at) + (lane % C::MB) * 16;
                page[i] = j < seg.kmax ? table[j >> p.pool.page_shift] : 0;
                return;
            }
            segment(p);
        }
    }
    static constexpr int CH = C::RB / 16;  // chunks per row
    static constexpr bool EVEN = (CH & (CH - 1)) == 0 && CH <= 32;
    // offset in a slot of the lane's i-th chunk of a block of 16 rows: a part by lane, and
    // a constant one
    __device__ static uint32_t place(int lane, int i)
    {
        if constexpr (EVEN) {
            const int r = lane / CH, c = lane % CH;
            return (r * C::RBS + ((c ^ C::key(r)) << 4)) ^ (C::key(i * (32 / CH)) << 4);
        } else {
            const int x = lane + 32 * i, r = x / CH, c = x - r * CH;
            return r * C::RBS + ((c ^ C::key(r)) << 4);
        }
    }
    __host__ __device__ static constexpr int place_more(int i) { return EVEN ? i * (32 / CH) * C::RBS : 0; }
    template <int MBI, int... I>
    __device__ static void block_whole(uint32_t dst, const uint8_t* rows, int lane, std::integer_sequence<int, I...>)
    {
        (copy16<MBI * 16 * C::RBS + place_more(I), I * 512>(dst + place(lane, I), rows), ...);
    }
    template <int... MBI>
    __device__ void step_whole(const uint8_t* pool, int lane, std::integer_sequence<int, MBI...>)
    {
        (block_whole<MBI>(slot, pool + off[MBI], lane, std::make_integer_sequence<int, CH / 2>{}), ...);
    }
    // the pairs of all the step's blocks: MB * SCB chunks
    template <int... I>
    __device__ void pairs_whole(const uint8_t* pool, int lane, std::integer_sequence<int, I...>)
    {
        constexpr int ALL = C::MB * C::SCB;
        auto from = [&](int i) {
            const int x = lane + 32 * i, mb = C::SCB % 32 == 0 ? i / (C::SCB / 32) : x / C::SCB;
            long long o = off[0] + poff[0];
            if (mb > 0) o = off[C::MB - 1] + poff[C::MB - 1] - C::SCB * 16;
            return pool + o;
        };
        static_assert(C::MB <= 2, "two blocks");
        ((lane + 32 * I < ALL ? copy16<C::TS * C::RBS + I * 512, I * 512>(slot + lane * 16, from(I)) : void()), ...);
    }

    template <bool VALUE>
    __device__ void issue(const PagedFwdParams& p)
    {
        const int lane = threadIdx.x & 31;
        if (base[0] >= 0) {
            if constexpr (!VALUE) {
                const bool good = static_cast<uint32_t>(page[0]) < static_cast<uint32_t>(p.pool.num_pages);
                bits = __ballot_sync(0xffffffffu, good) & ((1u << C::MB) - 1u);
                if (!good) record_bad_page(PAGED_FWD);
                // blocks are at least 1280 bytes, so a pool has fewer than 2^32 of them
                const uint32_t blk = good ? static_cast<uint32_t>(page[0]) * p.pool.Hkv + hkv[0] : 0u;
#pragma unroll
                for (int mb = 0; mb < C::MB; ++mb) {
                    const int slot0 = (base[0] + mb * 16) & (p.pool.page_size - 1);
                    off[mb] = static_cast<unsigned long long>(__shfl_sync(0xffffffffu, blk, mb)) * p.block_bytes + slot0 * C::RB;
                    poff[mb] = p.pool.page_size * C::RB - slot0 * (C::RB - C::SCB);
                }
                if (lane == 0) asm volatile("st.shared.b32 [%0], %1;" ::"r"(ok + 4u * n), "r"(bits) : "memory");
            }
            const uint8_t* const pool = static_cast<const uint8_t*>(VALUE ? p.v_cache : p.k_cache) + lane * 16;
            if (kmax[0] - base[0] >= C::TS && bits == (1u << C::MB) - 1u) {
                step_whole(pool, lane, std::make_integer_sequence<int, C::MB>{});
                if constexpr (INT4) pairs_whole(pool, lane, std::make_integer_sequence<int, (C::MB * C::SCB + 31) / 32>{});
            } else {
                // only what exists is read; the rest of the slot is zeros
#pragma unroll
                for (int mb = 0; mb < C::MB; ++mb) {
                    const uint32_t dst = slot + mb * 16 * C::RBS;
                    const uint8_t* const rows = pool + off[mb];
                    const int valid = (bits >> mb & 1u) ? max(0, min(16, kmax[0] - base[0] - mb * 16)) : 0;
#pragma unroll
                    for (int i = 0; i < CH / 2; ++i) {
                        const int left = max(0, min(16, valid * C::RB - (lane + 32 * i) * 16));
                        copy16_part(dst + place(lane, i) + place_more(i), left > 0 ? rows + i * 512 : pool, left);
                    }
                    if constexpr (INT4) {
                        const uint32_t pdst = slot + C::TS * C::RBS + mb * 16 * C::SCB + lane * 16;
#pragma unroll
                        for (int i = 0; i < (C::SCB + 31) / 32; ++i) {
                            const int left = max(0, min(16, valid * C::SCB - (lane + 32 * i) * 16));
                            if (lane + 32 * i < C::SCB)
                                copy16_part(pdst + i * 512, left > 0 ? rows + poff[mb] + i * 512 : pool, left);
                        }
                    }
                }
            }
            if constexpr (VALUE) {
                base[0] = base[1];
                kmax[0] = kmax[1];
                hkv[0] = hkv[1];
                page[0] = page[1];
                fetch(p, 1);
            }
        }
        copy_commit();
        slot += C::SLOT;
        if (++n == C::NST) {
            n = 0;
            slot -= C::NST * C::SLOT;
        }
    }
};

// ---------------------------------------------------------------------------------
// Q of a unit into shared memory, as the B fragments of the score products.
// ---------------------------------------------------------------------------------
template <int D, bool BF16, bool INT4, int NT>
__device__ __forceinline__ void paged_stage_q(const PagedFwdParams& p, const PagedSegment& x, uint8_t* to)
{
    using C = PagedCfg<D, INT4, NT>;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, gg = lane >> 2, t = lane & 3;
    const int h0 = p.by_hkv.remainder(x.u) * p.group;
    // the warps of a tile share its blocks of 32 dims
    static_assert(C::W % NT == 0, "warps per tile");
    constexpr int PER = C::W / NT;
    const int nt = w % NT, k0 = w / NT;
    const int r = x.r0 + nt * 8 + gg;
    const int tok = p.by_group.quotient(r);
    const bool ok = r < x.R;
    const uint16_t* src = static_cast<const uint16_t*>(p.q) +
                          (static_cast<size_t>(x.s.q0 + (ok ? tok : 0)) * p.Hq + h0 + (ok ? r - tok * p.group : 0)) * D;
    uint4* dst = reinterpret_cast<uint4*>(to) + nt * (D / 32) * 32 + lane;
    if constexpr (!INT4) {
#pragma unroll 4
        for (int k = k0; k < D / 32; k += PER) {  // two steps of 16 dims
            const uint32_t* s = reinterpret_cast<const uint32_t*>(src + k * 32) + t;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (ok) v = make_uint4(s[0], s[4], s[8], s[12]);
            dst[k * 32] = v;
        }
    } else {
        // dims 8 t .. 8 t + 7 of each group: pairs (i, i + 4).  Read twice: O is live here
        auto dims = [&](int k, float (&f)[8]) {
            pg_unpack8<BF16>(ok ? reinterpret_cast<const uint4*>(src + k * 32)[t] : make_uint4(0u, 0u, 0u, 0u), f);
        };
        float big = 0.0f;
#pragma unroll 8
        for (int k = 0; k < D / 32; ++k) {
            float f[8];
            dims(k, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) big = fmaxf(big, fabsf(f[i]));
        }
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        // the row's power of two: its largest value comes to 2^62 (bf16) or 2^14 (fp16)
        const int ex = static_cast<int>(__float_as_uint(big) >> 23) - 127;
        const int kq = BF16 ? max(7, min(100, 62 - ex)) : max(-2, min(38, 14 - ex));
        const float up = __uint_as_float(static_cast<uint32_t>(kq + 127) << 23);
        // the codes are 2^-133 (bf16) or 2^-24 (fp16) small
        const int dn = (BF16 ? 133 : 24) - kq;  // 33 .. 126 or -14 .. 26
        const float down = __uint_as_float(static_cast<uint32_t>(127 - dn) << 23);
#pragma unroll 4
        for (int k = k0; k < D / 32; k += PER) {
            float f[8], sum = 0.0f;
            dims(k, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += f[i];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (t == 0) reinterpret_cast<float*>(to + C::OFF_QS)[(nt * (D / 32) + k) * 8 + gg] = sum * down;
            uint32_t b[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = (i & 1) ? up * 0.0625f : up;
                b[i] = pg_pack2<BF16>(f[i] * u, f[i + 4] * u);
            }
            dst[k * 32] = make_uint4(b[0], b[1], b[2], b[3]);
        }
        // the score's factor undoes both
        if (t == 0 && k0 == 0)
            reinterpret_cast<float*>(to + C::OFF_F)[nt * 8 + gg] = p.sl2 * __uint_as_float(static_cast<uint32_t>(dn + 127) << 23);
    }
}

// ---------------------------------------------------------------------------------
// The second product where its tokens' values are not finite and not every row sees
// them: a token at a time, only what a row sees.  Rare; kept out of the way of the rest.
// ---------------------------------------------------------------------------------
// The mma row of a score tile that holds token (row & 7): at the narrowest rows the
// tokens are dealt so that the value loads of a warp meet no bank twice.
template <bool INT4, class C>
__device__ __forceinline__ int token_of_slot(int slot)
{
    return C::RBS == 64 && INT4 ? (slot & ~3) | ((slot & 1) << 1) | ((slot >> 1) & 1) : slot;
}

// Whether a slot's values hold an infinity or a NaN.  4 bits: whether a pair makes the
// lowest or the highest code one (finite fp16 pairs can: 8736 * 15 - 65504 = 65536); the
// other codes lie between.
template <int D, bool BF16, bool INT4, class C>
__device__ __forceinline__ bool paged_slot_bad(const uint8_t* vs)
{
    constexpr int BYTES = INT4 ? C::TS * C::SCB : C::TS * C::RBS;
    constexpr uint32_t EXP = BF16 ? 0x7f80u : 0x7c00u;
    const uint8_t* const from = INT4 ? vs + C::TS * C::RBS : vs;
    bool bad = false;
#pragma unroll 1
    for (int i = (threadIdx.x & 31) * 4; i < BYTES; i += 128) {
        uint32_t w = lds<uint32_t>(from + i);
        if constexpr (INT4) {
            const float2 sz = pg_unpack2<BF16>(w);
            w = pg_pack2<BF16>(sz.y, fmaf(15.0f, sz.x, sz.y));
        }
        bad |= (w & EXP) == EXP || (w >> 16 & EXP) == EXP;
    }
    return __any_sync(0xffffffffu, bad);
}

template <int D, bool BF16, bool INT4, int NT, class C>
__device__ __forceinline__ void paged_product_by_token(const uint8_t* vs, int base, uint32_t bits, const int (&lim)[NT][2],
                                                       const uint32_t (&ph)[C::MB][NT][2],
                                                       const uint32_t (&pl)[C::MB][NT][2], float (&o)[D / 16][NT][4])
{
    const int lane = threadIdx.x & 31, gg = lane >> 2, t = lane & 3;
#pragma unroll 1
    for (int k = 0; k < C::TS; ++k) {
        const int mb = k >> 4, row = mb * 16 + (k & 8) + token_of_slot<INT4, C>(k & 7);
        float w[NT][2];
        bool sees[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint32_t hi = (k & 8) ? ph[0][nt][1] : ph[0][nt][0], lo = (k & 8) ? pl[0][nt][1] : pl[0][nt][0];
            if (C::MB == 2 && mb) {
                hi = (k & 8) ? ph[C::MB - 1][nt][1] : ph[C::MB - 1][nt][0];
                lo = (k & 8) ? pl[C::MB - 1][nt][1] : pl[C::MB - 1][nt][0];
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // the weight of column 2 t + i lies with the lane that feeds it to the product
                const int from = (2 * t + i) * 4 + ((k & 7) >> 1);
                const float2 a = pg_unpack2<BF16>(__shfl_sync(0xffffffffu, hi, from));
                const float2 b = pg_unpack2<BF16>(__shfl_sync(0xffffffffu, lo, from));
                w[nt][i] = (k & 1) ? a.y + b.y : a.x + b.x;
                sees[nt][i] = (bits >> mb & 1u) && base + row < lim[nt][i];
            }
        }
        auto add = [&](int mt, float u, float v) {  // dims of the lane's rows of tile mt
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (sees[nt][i]) {
                        o[mt][nt][i] = fmaf(w[nt][i], u, o[mt][nt][i]);
                        o[mt][nt][2 + i] = fmaf(w[nt][i], v, o[mt][nt][2 + i]);
                    }
        };
        if constexpr (!INT4) {
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                const uint8_t* const at = vs + row * C::RBS + gg * 2;
                const uint16_t u = lds<uint16_t>(at + (((2 * mt) ^ C::key(row)) << 4));
                const uint16_t v = lds<uint16_t>(at + (((2 * mt + 1) ^ C::key(row)) << 4));
                add(mt, pg_unpack2<BF16>(u).x, pg_unpack2<BF16>(v).x);
            }
        } else {
#pragma unroll
            for (int ws = 0; ws < D / 64; ++ws) {
                const int c = 2 * ws + (gg >> 2);
                const uint32_t word = lds<uint32_t>(vs + row * C::RBS + ((c ^ C::key(row)) << 4) + (gg & 3) * 4);
                const float2 sz = pg_unpack2<BF16>(lds<uint32_t>(vs + C::TS * C::RBS + row * C::SCB + c * 4));
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float u = fmaf(static_cast<float>(word >> (4 * j) & 15u), sz.x, sz.y);
                    const float v = fmaf(static_cast<float>(word >> (16 + 4 * j) & 15u), sz.x, sz.y);
                    const float2 r = pg_unpack2<BF16>(pg_pack2<BF16>(u, v));
                    add(ws * 4 + j, r.x, r.y);
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------------
// What an output is that did not come out finite.  An infinity among the values times a
// weight in two terms is a NaN where the second is 0 or negative, or where the weight is
// too small for 32 bits; by the definition (a finite score's weight is above 0) it stays
// that infinity.  So the answer depends on no weight: +infinity, -infinity, or a NaN where
// the row sees one or both signs.  Looking at the values of every tile would cost each
// step; this looks at a row's again after the range, only where an output calls for it.
// Out of line and after the loop, where its registers are free, it costs calls without
// infinities 0 to 1 % (d = 512: 2 %); within the loop it cost 1 to 10 %.
// ---------------------------------------------------------------------------------
struct PagedValues {
    const uint8_t* pool;  // of the KV head, at page 0
    const int* table;     // of the sequence
    size_t page_bytes;    // from one page to the next
    int shift, num_pages;
};
// For dims 8 v .. 8 v + 7 of the tokens from .. to - 1 (from: a multiple of 16) two bits
// each: 1 if one of them is +infinity, 2 if one is -infinity, 3 for both or a NaN.
template <int D, bool BF16, bool INT4>
__device__ uint32_t paged_not_finite(const PagedValues& at, int from, int to, int v)
{
    constexpr uint32_t EXP = BF16 ? 0x7f80u : 0x7c00u;
    constexpr int RB = INT4 ? D / 2 : 2 * D;
    uint32_t found = 0;
    for (long long j = from; j < to && found != 0xffffu; j += 16) {
        const int page = at.table[j >> at.shift];
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(at.num_pages)) continue;
        const int slot = static_cast<int>(j) & ((1 << at.shift) - 1), n = static_cast<int>(min(16ll, to - j));
        const uint8_t* const block = at.pool + page * at.page_bytes;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const uint8_t* const row = block + static_cast<size_t>(slot + i) * RB;
            const uint4 x = read_vector<D, BF16, INT4>(row, block + (static_cast<size_t>(RB) << at.shift) + (slot + i) * (D / 8), v);
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t y = k & 1 ? u[k / 2] >> 16 : u[k / 2] & 0xffffu;
                if ((y & EXP) == EXP) found |= ((y & 0x7fffu) != EXP ? 3u : y & 0x8000u ? 2u : 1u) << (2 * k);
            }
        }
    }
    return found;
}

// A range's outputs (or pieces of them) as the join of the warps has written them: the
// same thread looks at what it wrote.
template <int D, bool BF16, bool INT4, int NT>
__device__ __noinline__ void paged_settle(const PagedFwdParams& p, const PagedStart& start)
{
    using C = PagedCfg<D, INT4, NT>;
    PagedWalk<C> walk;
    PagedSegment x;
    walk.init(p, start);
    while (walk.next(p, x)) {
        const bool whole = x.first && x.last;
        const size_t piece = (2 * static_cast<size_t>(blockIdx.x) + (x.first ? 1 : 0)) * C::ROWS;
        const int hkv = p.by_hkv.remainder(x.u);
        const PagedValues at{static_cast<const uint8_t*>(p.v_cache) + static_cast<size_t>(hkv) * p.block_bytes,
                             p.pool.table + static_cast<size_t>(x.b) * p.pool.max_pages,
                             static_cast<size_t>(p.block_bytes) * p.pool.Hkv, p.pool.page_shift, p.pool.num_pages};
#pragma unroll 1
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll 1
            for (int part = 0; part < D / C::DP; ++part) {
#pragma unroll 1
                for (int y = threadIdx.x; y < C::DP; y += C::THREADS) {
                    const int rr = y / (C::DP / 8), v = part * (C::DP / 8) + y - rr * (C::DP / 8), r = x.r0 + nt * 8 + rr;
                    if (r >= x.R) continue;
                    const int tok = p.by_group.quotient(r), h = hkv * p.group + r - tok * p.group;
                    uint16_t* const o = static_cast<uint16_t*>(p.o) + (static_cast<size_t>(x.s.q0 + tok) * p.Hq + h) * D + v * 8;
                    float* const partial = p.opart + (piece + nt * 8 + rr) * D + v * 8;
                    const float sum = whole ? p.lse[static_cast<size_t>(h) * p.total_q + x.s.q0 + tok] : p.mlpart[piece + nt * 8 + rr].y;
                    float acc[8], odd = 0.0f;
                    if (whole) pg_unpack8<BF16>(*reinterpret_cast<const uint4*>(o), acc);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        if (!whole) acc[i] = partial[i];
                        odd = fmaf(acc[i], 0.0f, odd);
                    }
                    if (!(odd != 0.0f) || !isfinite(sum)) continue;
                    // the row's tokens among the segment's
                    const long long seen = p.causal ? min(x.s.Sk, tok + x.s.Sk - x.s.Sq + 1) : x.s.Sk;
                    const long long end = min(static_cast<long long>(x.g1) * C::GR, seen);
                    const uint32_t found = paged_not_finite<D, BF16, INT4>(
                        at, static_cast<int>(min(static_cast<long long>(x.g0) * C::GR, end)), static_cast<int>(end), v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t is = found >> (2 * i) & 3u;
                        if (is) acc[i] = is == 3u ? NAN : is == 1u ? INFINITY : -INFINITY;
                        if (!whole) partial[i] = acc[i];
                    }
                    if (whole) *reinterpret_cast<uint4*>(o) = pg_pack8<BF16>(acc);
                }
            }
        }
    }
}

// ---------------------------------------------------------------------------------
// The kernel
// ---------------------------------------------------------------------------------
template <int D, bool BF16, bool INT4, int NT>
__global__ void __launch_bounds__(PagedCfg<D, INT4, NT>::THREADS, PagedCfg<D, INT4, NT>::CTAS)
    fa_fwd_paged_kernel(const __grid_constant__ PagedFwdParams p)
{
    using C = PagedCfg<D, INT4, NT>;
    constexpr int MB = C::MB;
    constexpr int MT = D / 16;  // 16-dim tiles of O^T
    constexpr float UP = BF16 ? 0.0f : 14.0f, SLACK = BF16 ? 8.0f : 1.0f;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ PagedStart start;
    __shared__ long long red[33];
    __shared__ int unsettled;  // whether an output of the range is not finite though its weights are
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, gg = lane >> 2, t = lane & 3;
    const uint32_t sbase = smem_u32(smem);
    if (threadIdx.x == 0) unsettled = 0;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    paged_start<C>(p, &start, red);
    if (threadIdx.x == 0 && p.rec != nullptr) p.rec[blockIdx.x].last = -1;
    if (start.lo >= start.hi) {
        if (p.rec != nullptr && threadIdx.x < C::ROWS)
            p.mlpart[2 * static_cast<size_t>(blockIdx.x) * C::ROWS + threadIdx.x] = make_float2(-INFINITY, 0.0f);
        return;
    }

    const uint32_t ring = sbase + C::OFF_RING + w * C::NST * C::SLOT;
    const uint32_t okw = sbase + C::OFF_OK + w * 32;
    PagedLoad<D, INT4, NT> load;
    load.init(p, start, ring, okw);
#pragma unroll
    for (int i = 0; i < C::NST - 1; ++i) {
        if (i & 1) load.template issue<true>(p);
        else load.template issue<false>(p);
    }
    constexpr bool AHEAD = (C::NST - 1) & 1;  // NST - 1 copies ahead of a key tile: a value tile
    uint32_t n = 0, at = C::OFF_RING + w * C::NST * C::SLOT;  // the slot consumed next, and its offset
    auto turn = [&] {
        at += C::SLOT;
        if (++n == C::NST) {
            n = 0;
            at -= C::NST * C::SLOT;
        }
    };

    auto tok_of = [](int slot) { return token_of_slot<INT4, C>(slot); };
    const int row_a = tok_of(gg);
    // offsets in a slot of the lane's key words (rows row_a, row_a + 8) and value words
    // (rows v_row, the next slot's token, and both + 8)
    const uint32_t key_a = row_a * C::RBS + (C::key(row_a) << 4) + t * 4;
    const int v_row = tok_of(2 * t);
    constexpr int V_NEXT = C::RBS == 64 ? 2 : 1;  // tok_of(2 t + 1) - tok_of(2 t); changes key() by 1
    const uint32_t val_a = v_row * C::RBS + (((gg >> 2) ^ C::key(v_row)) << 4) + (gg & 3) * 4;
    const uint32_t pair_a = v_row * C::SCB + (gg >> 2) * 4;

    PagedWalk<C> walk;
    walk.init(p, start);
    PagedSegment x, following;
    bool more = walk.next(p, x);  // the range is not empty
    uint32_t turns = 0;           // which of the two places for Q and for (m, l)
    paged_stage_q<D, BF16, INT4, NT>(p, x, smem + C::OFF_Q);
    __syncthreads();
    for (; more; x = following, turns ^= 1u) {
        const uint8_t* const sq = smem + C::OFF_Q + turns * C::Q_BYTES;
        float o[MT][NT][4];
        float m[NT][2], l[NT][2], f[NT][2];
        int lim[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[nt][i] = -INFINITY;
                l[nt][i] = 0.0f;
                const int r = x.r0 + nt * 8 + 2 * t + i;
                f[nt][i] = INT4 ? reinterpret_cast<const float*>(sq + C::OFF_F)[nt * 8 + 2 * t + i] : p.sl2;
                lim[nt][i] = p.causal && r < x.R ? min(x.s.Sk, p.by_group.quotient(r) + x.s.Sk - x.s.Sq + 1) : x.s.Sk;
            }
        }
        const int lim0 = p.causal ? min(x.s.Sk, p.by_group.quotient(x.r0) + x.s.Sk - x.s.Sq + 1) : x.s.Sk;  // the least

        for (int g = x.g0; g < x.g1; ++g) {
            const uint32_t at0 = static_cast<uint32_t>(g) * C::GR + w * C::TS;
            if (at0 >= static_cast<uint32_t>(x.kmax)) break;
            const int base = static_cast<int>(at0);
            // ---- scores
            copy_wait<C::NST - 2>();
            __syncwarp();
            load.template issue<AHEAD>(p);  // into the slot consumed last
            const uint32_t kat = at;
            const uint8_t* const ks = smem + kat;
            const uint32_t bits = lds<uint32_t>(smem + C::OFF_OK + (w * 8 + n) * 4);
            turn();
            float s[MB][NT][4];
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[mb][nt][i] = 0.0f;
            if constexpr (!INT4) {
                const int r = lane & 15;
                const uint32_t row = sbase + kat + r * C::RBS;
#pragma unroll
                for (int k = 0; k < D / 32; ++k) {
                    uint32_t a0[4], a1[4];
                    const int c = 4 * k + (lane >> 4);
                    ldmatrix4(a0, row + ((c ^ (r & 7)) << 4));
                    ldmatrix4(a1, row + (((c + 2) ^ (r & 7)) << 4));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint4 b = lds<uint4>(sq + ((nt * (D / 32) + k) * 32 + lane) * 16);
                        mma16816<BF16>(s[0][nt], a0, b.x, b.y);
                        mma16816<BF16>(s[0][nt], a1, b.z, b.w);
                    }
                }
            } else {
#pragma unroll 1
                for (int k4 = 0; k4 < D / 32; k4 += (D % 128 == 0 ? 4 : 2)) {
                    constexpr int KG = D % 128 == 0 ? 4 : 2;  // groups per load of pairs
                    uint32_t pr[MB][2][KG];
#pragma unroll
                    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                        for (int y = 0; y < 2; ++y) {
                            const uint8_t* a = ks + row_a * C::SCB + (C::TS * C::RBS + (mb * 16 + y * 8) * C::SCB + k4 * 4);
                            if constexpr (KG == 4) {
                                const uint4 v = lds<uint4>(a);
                                pr[mb][y][0] = v.x;
                                pr[mb][y][1] = v.y;
                                pr[mb][y][2] = v.z;
                                pr[mb][y][3] = v.w;
                            } else {
                                const uint2 v = lds<uint2>(a);
                                pr[mb][y][0] = v.x;
                                pr[mb][y][1] = v.y;
                            }
                        }
#pragma unroll
                    for (int kk = 0; kk < KG; ++kk) {
                        const int k = k4 + kk;
                        uint4 b[NT];
                        float2 qs[NT];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            b[nt] = lds<uint4>(sq + ((nt * (D / 32) + k) * 32 + lane) * 16);
                            qs[nt] = lds<float2>(sq + C::OFF_QS + ((nt * (D / 32) + k) * 8 + 2 * t) * 4);
                        }
#pragma unroll
                        for (int mb = 0; mb < MB; ++mb) {
                            const uint8_t* const wk = ks + (key_a ^ ((k & C::LINE) << 4)) +
                                                      (((k * 16) & ~(C::LINE * 16 + 15)) + mb * 16 * C::RBS);
                            const uint32_t wa = lds<uint32_t>(wk), wb = lds<uint32_t>(wk + 8 * C::RBS);
                            const uint32_t a0[4] = {code_tiny<false>(wa), code_tiny<false>(wb), code_tiny<true>(wa), code_tiny<true>(wb)};
                            const uint32_t a1[4] = {code_tiny<false>(wa >> 8), code_tiny<false>(wb >> 8), code_tiny<true>(wa >> 8),
                                                    code_tiny<true>(wb >> 8)};
                            const float2 za = pg_unpack2<BF16>(pr[mb][0][kk]), zb = pg_unpack2<BF16>(pr[mb][1][kk]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                float d[4];
                                mma16816_first<BF16>(d, a0, b[nt].x, b[nt].y);
                                mma16816<BF16>(d, a1, b[nt].z, b[nt].w);
                                s[mb][nt][0] = fmaf(za.x, d[0], fmaf(za.y, qs[nt].x, s[mb][nt][0]));
                                s[mb][nt][1] = fmaf(za.x, d[1], fmaf(za.y, qs[nt].y, s[mb][nt][1]));
                                s[mb][nt][2] = fmaf(zb.x, d[2], fmaf(zb.y, qs[nt].x, s[mb][nt][2]));
                                s[mb][nt][3] = fmaf(zb.x, d[3], fmaf(zb.y, qs[nt].y, s[mb][nt][3]));
                            }
                        }
                    }
                }
            }
            // ---- the scale, in base 2.  Rounded here, once: a difference to the rounded maximum
            // is then never above the true one's sign, however large the scores are
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[mb][nt][i] *= f[nt][i & 1];
            // ---- masks: causal limits, the sequence's end, tokens without a page
            const bool whole = (bits & ((1u << MB) - 1u)) == (1u << MB) - 1u;
            if (base > lim0 - C::TS || !whole) {
#pragma unroll
                for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const int j = base + mb * 16 + y * 8 + row_a;
                        const bool has = bits >> mb & 1u;
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (!has || j >= lim[nt][i]) s[mb][nt][2 * y + i] = -INFINITY;
                    }
            }
            // ---- online softmax; columns 2 t, 2 t + 1 of each tile
            bool grow = false;
            float mx[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float v = fmaxf(s[0][nt][i], s[0][nt][2 + i]);
#pragma unroll
                    for (int mb = 1; mb < MB; ++mb) v = fmaxf(v, fmaxf(s[mb][nt][i], s[mb][nt][2 + i]));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    mx[nt][i] = v;
                    grow |= BF16 ? mx[nt][i] > m[nt][i] + SLACK : mx[nt][i] - m[nt][i] > UP + SLACK;
                }
            // the reference (m) lies UP below the greatest score met when it last moved.  It moves
            // (and O and l with it) only when a score exceeds it by more than UP + SLACK, so weights
            // reach 2^8 in bf16 and 2^15 in fp16.  The most that fp16 allows (UP 7 and SLACK 8: 128 times
            // coarser, and no faster: 4 sequences of 131,072 tokens, d = 256, 166.0 us against 165.8;
            // 4-bit, d = 128, 103.3 against 103.9)
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float al[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float ref = mx[nt][i] - UP;
                        // scores past 2^26 are further apart than UP: the difference was rounded
                        if (!BF16 && mx[nt][i] - ref > UP + SLACK) ref = mx[nt][i];
                        const float mn = fmaxf(m[nt][i], ref);
                        al[i] = m[nt][i] == mn ? 1.0f : ex2_sfu(m[nt][i] - mn);
                        m[nt][i] = mn;
                        l[nt][i] *= al[i];
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[mt][nt][i] *= al[i & 1];
                }
            }
            // ---- P, in two 16-bit terms, as the B fragments of the second product
            uint32_t ph[MB][NT][2], pl[MB][NT][2];
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        float v[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const float ref = m[nt][i] == -INFINITY ? 0.0f : m[nt][i];
                            v[i] = ex2_sfu(s[mb][nt][2 * y + i] - ref);
                            l[nt][i] += v[i];
                        }
                        const uint32_t hi = pg_pack2<BF16>(v[0], v[1]);
                        const float2 b = pg_unpack2<BF16>(hi);
                        ph[mb][nt][y] = transpose8x8(hi);
                        pl[mb][nt][y] = transpose8x8(pg_pack2<BF16>(v[0] - b.x, v[1] - b.y));
                    }
            // ---- O^T += V^T P^T
            copy_wait<C::NST - 2>();
            __syncwarp();
            load.template issue<!AHEAD>(p);
            const uint32_t vat = at;
            const uint8_t* const vs = smem + vat;
            turn();
            // Where some rows see a token and others do not, an infinity or a NaN among its
            // values must not meet the others' weight of 0 in a product
            bool plain = true;
            if (base > lim0 - C::TS && lim0 < x.kmax) plain = !paged_slot_bad<D, BF16, INT4, C>(vs);
            if (!plain) {
                paged_product_by_token<D, BF16, INT4, NT, C>(vs, base, bits, lim, ph, pl, o);
            } else if constexpr (!INT4) {
                const int r = (lane & 7) + ((lane >> 4) << 3);
                const uint32_t row = sbase + vat + r * C::RBS;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t a[4];
                    ldmatrix4_trans(a, row + (((2 * mt + ((lane >> 3) & 1)) ^ (r & 7)) << 4));
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816<BF16>(o[mt][nt], a, ph[0][nt][0], ph[0][nt][1]);
                        mma16816<BF16>(o[mt][nt], a, pl[0][nt][0], pl[0][nt][1]);
                    }
                }
            } else {
#pragma unroll
                for (int mb = 0; mb < MB; ++mb) {
#pragma unroll
                    for (int ws = 0; ws < D / 64; ++ws) {  // 64 dims: word gg of eight
                        uint32_t wd[4], pr[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = mb * 16 + (i & 1) * V_NEXT + (i >> 1) * 8;
                            wd[i] = lds<uint32_t>(vs + (val_a ^ ((((2 * ws) & C::LINE) ^ (i & 1)) << 4)) +
                                                  (row * C::RBS + ((2 * ws * 16) & ~(C::LINE * 16 + 15))));
                            pr[i] = lds<uint32_t>(vs + pair_a + (C::TS * C::RBS + row * C::SCB + ws * 8));
                        }
                        const uint32_t lo01 = __byte_perm(wd[0], wd[1], 0x5410), hi01 = __byte_perm(wd[0], wd[1], 0x7632);
                        const uint32_t lo23 = __byte_perm(wd[2], wd[3], 0x5410), hi23 = __byte_perm(wd[2], wd[3], 0x7632);
                        const uint32_t s01 = __byte_perm(pr[0], pr[1], 0x5410), z01 = __byte_perm(pr[0], pr[1], 0x7632);
                        const uint32_t s23 = __byte_perm(pr[2], pr[3], 0x5410), z23 = __byte_perm(pr[2], pr[3], 0x7632);
                        uint32_t s01q = s01, s23q = s23;
                        if constexpr (BF16) {
                            s01q = mul_bf16x2(s01, 0x40804080u);
                            s23q = mul_bf16x2(s23, 0x40804080u);
                        }
                        // tile j of the 64 dims: rows gg and gg + 8 are dims j and 4 + j of the word
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int sh = (j >> 1) * 8;
                            uint32_t a[4];
                            if (j & 1) {
                                a[0] = code_value<BF16, true>(lo01 >> sh, s01, s01q, z01);
                                a[1] = code_value<BF16, true>(hi01 >> sh, s01, s01q, z01);
                                a[2] = code_value<BF16, true>(lo23 >> sh, s23, s23q, z23);
                                a[3] = code_value<BF16, true>(hi23 >> sh, s23, s23q, z23);
                            } else {
                                a[0] = code_value<BF16, false>(lo01 >> sh, s01, s01q, z01);
                                a[1] = code_value<BF16, false>(hi01 >> sh, s01, s01q, z01);
                                a[2] = code_value<BF16, false>(lo23 >> sh, s23, s23q, z23);
                                a[3] = code_value<BF16, false>(hi23 >> sh, s23, s23q, z23);
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma16816<BF16>(o[ws * 4 + j][nt], a, ph[mb][nt][0], ph[mb][nt][1]);
                                mma16816<BF16>(o[ws * 4 + j][nt], a, pl[mb][nt][0], pl[mb][nt][1]);
                            }
                        }
                    }
                }
            }
        }

        // ---- the warps' pieces of the unit become one
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float v = l[nt][i];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (gg == 0)
                    reinterpret_cast<float2*>(smem + C::OFF_ML)[(turns * C::W + w) * C::ROWS + nt * 8 + 2 * t + i] = make_float2(m[nt][i], v);
            }
        more = walk.next(p, following);
        if (more) paged_stage_q<D, BF16, INT4, NT>(p, following, smem + C::OFF_Q + (turns ^ 1u) * C::Q_BYTES);
        __syncthreads();
        const float2* const ml = reinterpret_cast<const float2*>(smem + C::OFF_ML) + turns * C::W * C::ROWS;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float top = -INFINITY;
#pragma unroll
                for (int v = 0; v < C::W; ++v) top = fmaxf(top, ml[v * C::ROWS + nt * 8 + 2 * t + i].x);
                const float al = m[nt][i] == -INFINITY ? 0.0f : ex2_sfu(m[nt][i] - top);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    o[mt][nt][i] *= al;
                    o[mt][nt][2 + i] *= al;
                }
            }
        const bool whole = x.first && x.last;
        const size_t piece = (2 * static_cast<size_t>(blockIdx.x) + (x.first ? 1 : 0)) * C::ROWS;
        const int h0 = p.by_hkv.remainder(x.u) * p.group;
        float* buf = reinterpret_cast<float*>(smem + C::OFF_RED);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int part = 0; part < D / C::DP; ++part) {
                if (nt + part > 0) __syncthreads();
#pragma unroll
                for (int y = 0; y < C::DP / 16; ++y)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        buf[(w * 8 + 2 * t + (i & 1)) * C::MP + y * 16 + (i >> 1) * 8 + gg] = o[part * (C::DP / 16) + y][nt][i];
                __syncthreads();
                // thread: row rr of the tile, eight neighbouring dims (word v of the part)
                for (int y = threadIdx.x; y < C::DP; y += C::THREADS) {
                    const int rr = y / (C::DP / 8), v = y - rr * (C::DP / 8), r = x.r0 + nt * 8 + rr;
                    if (r >= x.R) continue;
                    float acc[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
#pragma unroll
                    for (int ww = 0; ww < C::W; ++ww)
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            // place of dim 8 v + i of the part in the tiles
                            const int at = INT4 ? (v >> 3) * 64 + (i & 3) * 16 + (i >> 2) * 8 + (v & 7) : 8 * v + i;
                            acc[i] += buf[(ww * 8 + rr) * C::MP + at];
                        }
                    float top = -INFINITY, sum = 0.0f;
#pragma unroll
                    for (int ww = 0; ww < C::W; ++ww) top = fmaxf(top, ml[ww * C::ROWS + nt * 8 + rr].x);
#pragma unroll
                    for (int ww = 0; ww < C::W; ++ww) {
                        const float2 z = ml[ww * C::ROWS + nt * 8 + rr];
                        if (z.y != 0.0f) sum += z.y * ex2_sfu(z.x - top);  // a NaN stays one
                    }
                    // not finite if one of them is not
                    const float odd = ((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7]));
                    if (!isfinite(odd) && isfinite(sum)) unsettled = 1;
                    if (whole) {
                        const int tok = p.by_group.quotient(r), h = h0 + r - tok * p.group;
                        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                        for (int i = 0; i < 8; ++i) acc[i] *= inv;
                        reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) +
                                                 (static_cast<size_t>(x.s.q0 + tok) * p.Hq + h) * D + part * C::DP)[v] =
                            pg_pack8<BF16>(acc);
                        if (part == 0 && v == 0)
                            p.lse[static_cast<size_t>(h) * p.total_q + x.s.q0 + tok] =
                                sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
                    } else {
                        float4* dst = reinterpret_cast<float4*>(p.opart + (piece + nt * 8 + rr) * D + part * C::DP + v * 8);
                        dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
                        dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
                        if (part == 0 && v == 0) p.mlpart[piece + nt * 8 + rr] = make_float2(top, sum);
                    }
                }
            }
        }
        if (!whole && x.first && threadIdx.x == 0) {
            // the pieces that follow are in the ranges up to the one that holds the unit's end
            const long long end = start.hi + x.left;
            const long long last = divide(end * gridDim.x + start.total - 1, start.total) - 1;
            p.rec[blockIdx.x] = PagedRecord{x.b, x.u, static_cast<int>(last), 0};
        }
    }
    copy_wait<0>();
    __syncthreads();
    if (unsettled) paged_settle<D, BF16, INT4, NT>(p, start);
}

// ---------------------------------------------------------------------------------
// Joins the pieces of the units that were cut.  A block has one record; with few pieces
// each warp joins rows of its own, with many the warps of the block share a row's.  The
// order of every sum is fixed by the pieces' number.
// ---------------------------------------------------------------------------------
constexpr int kJoinWarps = 8;
constexpr int kJoinFew = 16;

// Adds pieces first, first + step, .. of a row; lane's dims lane + 32 c.
template <int D, int ROWS>
__device__ __forceinline__ void join_pieces(const PagedFwdParams& p, int last, int row, int first, int step,
                                            float (&acc)[D / 32], float& m, float& l)
{
    const int lane = threadIdx.x & 31;
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) acc[c] = 0.0f;
    for (int j0 = first; j0 <= last; j0 += 32 * step) {  // 32 pieces' statistics at a time
        auto piece = [&](int j) {
            return (2 * static_cast<size_t>(j) + (j == static_cast<int>(blockIdx.x) ? 1 : 0)) * ROWS + row;
        };
        const int j = j0 + lane * step;
        float2 z = make_float2(-INFINITY, 0.0f);
        if (j <= last) z = p.mlpart[piece(j)];
        float mn = z.x;
#pragma unroll
        for (int o = 16; o; o >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mn = fmaxf(mn, m);
        // at least the least number, so that an infinity among the pieces stays one
        const float a = l == 0.0f ? 0.0f : fmaxf(ex2_sfu(m - mn), FLT_MIN);
        const float b = z.y == 0.0f ? 0.0f : fmaxf(ex2_sfu(z.x - mn), FLT_MIN);
        float sum = z.y * b;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        m = mn;
        l = l * a + sum;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) acc[c] *= a;
        const uint32_t some = __ballot_sync(0xffffffffu, z.y != 0.0f);
        const int n = min(32, (last - j0) / step + 1);
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            if (!(some >> i & 1u)) continue;  // nothing was written
            const float f = __shfl_sync(0xffffffffu, b, i);
            const float* src = p.opart + piece(j0 + i * step) * D + lane;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) acc[c] = fmaf(src[32 * c], f, acc[c]);
        }
    }
}

template <int D, bool BF16, int ROWS>
__global__ void __launch_bounds__(kJoinWarps * 32) fa_fwd_paged_join_kernel(const __grid_constant__ PagedFwdParams p)
{
    __shared__ float part[kJoinWarps][D];
    __shared__ float2 ml[kJoinWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PagedRecord rec = p.rec[blockIdx.x];
    if (rec.last < 0) return;
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q0 = p.cu_q[rec.b];
    const int Sq = max(0, min(p.cu_q[rec.b + 1] - q0, p.max_q));
    const int r0 = p.by_hkv.quotient(rec.u) * ROWS, rows = min(ROWS, Sq * p.group - r0);
    const int h0 = p.by_hkv.remainder(rec.u) * p.group;
    float acc[D / 32], m, l;
    const bool few = gridDim.y == 1 && rec.last - static_cast<int>(blockIdx.x) < kJoinFew;
    for (int row = few ? w : blockIdx.y; row < rows; row += few ? kJoinWarps : gridDim.y) {
        const int tok = p.by_group.quotient(r0 + row), h = h0 + r0 + row - tok * p.group;
        uint16_t* const dst = static_cast<uint16_t*>(p.o) + (static_cast<size_t>(q0 + tok) * p.Hq + h) * D;
        float* const lse = p.lse + static_cast<size_t>(h) * p.total_q + q0 + tok;
        if (few) {
            join_pieces<D, ROWS>(p, rec.last, row, blockIdx.x, 1, acc, m, l);
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) dst[lane + 32 * c] = static_cast<uint16_t>(pg_pack2<BF16>(acc[c] * inv, 0.0f));
            if (lane == 0) *lse = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
            continue;
        }
        join_pieces<D, ROWS>(p, rec.last, row, blockIdx.x + w, kJoinWarps, acc, m, l);
        __syncthreads();  // the last row's parts are done with
#pragma unroll
        for (int c = 0; c < D / 32; ++c) part[w][lane + 32 * c] = acc[c];
        if (lane == 0) ml[w] = make_float2(m, l);
        __syncthreads();
        float top = -INFINITY, sum = 0.0f, f[kJoinWarps];
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) top = fmaxf(top, ml[i].x);
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) {
            f[i] = ml[i].y == 0.0f ? 0.0f : fmaxf(ex2_sfu(ml[i].x - top), FLT_MIN);
            sum += ml[i].y * f[i];
        }
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        for (int c = threadIdx.x; c < D / 2; c += kJoinWarps * 32) {
            float a = 0.0f, b = 0.0f;
#pragma unroll
            for (int i = 0; i < kJoinWarps; ++i) {
                a = fmaf(f[i], part[i][2 * c], a);
                b = fmaf(f[i], part[i][2 * c + 1], b);
            }
            reinterpret_cast<uint32_t*>(dst)[c] = pg_pack2<BF16>(a * inv, b * inv);
        }
        if (threadIdx.x == 0) *lse = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
    }
}

}  // namespace fa
