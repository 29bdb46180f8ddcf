// fa_paged.cu -- the paged-cache entry points declared in include/fa.h: argument checks
// and launches.  Every entry point validates first and launches nothing on an invalid
// argument.
#include <atomic>
#include <cmath>

#include "fa_host.h"
#include "fa_paged.cuh"
#include "fa_paged_fwd.cuh"

namespace fa {

cudaError_t paged_status_read(uint32_t (&h)[4], cudaStream_t s)
{
    return cudaMemcpyFromSymbolAsync(h, g_paged_status, sizeof(h), 0, cudaMemcpyDeviceToHost, s);
}

cudaError_t paged_status_clear(cudaStream_t s)
{
    static const uint32_t zero[4] = {0, 0, 0, 0};
    return cudaMemcpyToSymbolAsync(g_paged_status, zero, sizeof(zero), 0, cudaMemcpyHostToDevice, s);
}

}  // namespace fa

namespace {

using fa::aligned16;
using fa::device_info;
using fa::DeviceInfo;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool head_dim_ok(int d) { return d == 128 || d == 192 || d == 256 || d == 384 || d == 512; }

bool page_size_ok(int n) { return n == 16 || n == 32 || n == 64 || n == 128 || n == 256; }

// Checks shared by the three calls; fills the kernels' view of the pools.
fa_status check_pool(const void* k_cache, const void* v_cache, const int* table, int B, int Hkv, int d,
                     int page_size, int num_pages, int max_pages, fa_kv_format fmt, fa_dtype dt, fa::PoolView* v)
{
    if (!k_cache || !v_cache || !table) return FA_ERR_INVALID_ARG;
    if (B < 1 || Hkv < 1 || num_pages < 1 || max_pages < 1) return FA_ERR_INVALID_ARG;
    if (!head_dim_ok(d) || (dt != FA_BF16 && dt != FA_FP16) || (fmt != FA_KV_16 && fmt != FA_KV_INT4))
        return FA_ERR_UNSUPPORTED;
    if (!page_size_ok(page_size)) return FA_ERR_UNSUPPORTED;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned4(table)) return FA_ERR_INVALID_ARG;
    // token positions of a sequence are 32-bit
    if (static_cast<long long>(max_pages) * page_size >= (1LL << 31)) return FA_ERR_INVALID_ARG;
    int shift = 0;
    while ((1 << shift) < page_size) ++shift;
    *v = fa::PoolView{table, Hkv, page_size, shift, num_pages, max_pages};
    return FA_OK;
}

template <int D>
fa_status launch_append(const fa::AppendParams& p, unsigned blocks, bool bf16, bool int4, cudaStream_t s)
{
    if (int4) {
        if (bf16) fa::fa_kv_append_kernel<D, true, true><<<blocks, 256, 0, s>>>(p);
        else fa::fa_kv_append_kernel<D, false, true><<<blocks, 256, 0, s>>>(p);
    } else {
        if (bf16) fa::fa_kv_append_kernel<D, true, false><<<blocks, 256, 0, s>>>(p);
        else fa::fa_kv_append_kernel<D, false, false><<<blocks, 256, 0, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D>
fa_status launch_gather(const fa::GatherParams& p, unsigned blocks, bool bf16, bool int4, cudaStream_t s)
{
    if (int4) {
        if (bf16) fa::fa_kv_gather_kernel<D, true, true><<<blocks, 256, 0, s>>>(p);
        else fa::fa_kv_gather_kernel<D, false, true><<<blocks, 256, 0, s>>>(p);
    } else {
        if (bf16) fa::fa_kv_gather_kernel<D, true, false><<<blocks, 256, 0, s>>>(p);
        else fa::fa_kv_gather_kernel<D, false, false><<<blocks, 256, 0, s>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Eight-row tiles of a unit: the fewest that hold the rows of a sequence at once, as far
// as a warp's registers go (O^T takes NT * D / 4 of them).  A wider unit reads the pages
// for more rows at a time.
int paged_tiles(int max_q, int group, int d)
{
    const long long rows = static_cast<long long>(max_q) * group;
    const int most = d == 128 ? 4 : d <= 256 ? 2 : 1;
    int nt = 1;
    while (nt < most && 8 * nt < rows) nt *= 2;
    return nt;
}

// Resident CTAs of the forward's grid, at most.
int paged_grid_max(int sm_count) { return fa::kPagedCtas * sm_count; }

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t paged_workspace(int sm_count, int rows, int d, fa::PagedFwdParams* p, void* ws)
{
    const size_t n = paged_grid_max(sm_count);
    const size_t o = round256(2 * n * rows * d * 4), ml = round256(2 * n * rows * 8), rec = round256(n * sizeof(fa::PagedRecord));
    if (p) {
        uint8_t* w = static_cast<uint8_t*>(ws);
        p->opart = reinterpret_cast<float*>(w);
        p->mlpart = reinterpret_cast<float2*>(w + o);
        p->rec = reinterpret_cast<fa::PagedRecord*>(w + o + ml);
    }
    return o + ml + rec;
}

template <int D, bool BF16, bool INT4, int NT>
fa_status launch_paged(const fa::PagedFwdParams& p, int sm_count, cudaStream_t s)
{
    using C = fa::PagedCfg<D, INT4, NT>;
    auto kernel = fa::fa_fwd_paged_kernel<D, BF16, INT4, NT>;
    // once per device: the call is a noticeable part of a decode step's host time
    static std::atomic<uint64_t> ready{0};
    static_assert(fa::kMaxDevices <= 64, "one bit per device");
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= fa::kMaxDevices) return FA_ERR_CUDA;
    if (!(ready.load(std::memory_order_acquire) >> dev & 1u)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
            return FA_ERR_CUDA;
        ready.fetch_or(1ull << dev, std::memory_order_release);
    }
    // no more CTAs than there can be granules
    const long long blocks = (static_cast<long long>(p.max_q) * p.group + C::ROWS - 1) / C::ROWS;
    const long long keys = static_cast<long long>(p.pool.max_pages) << p.pool.page_shift;
    const double units = static_cast<double>(p.B) * blocks * p.pool.Hkv;
    const long long granules = (keys + C::GR - 1) / C::GR;
    int grid = C::CTAS * sm_count;
    // Few short sequences: a unit stays whole, and nothing is left to join.  Up to about
    // 160 KB of keys and values one CTA takes no longer than the pieces and their join (one
    // sequence, 8 KV heads, d = 128: 64 / 256 / 384 / 512 tokens 5.9 / 8.1 / 9.2 / 11.2 us
    // whole, 6.9 / 8.9 / 8.9 / 8.9 us in pieces), and a launch less is 2 us of host time.
    // The host knows the table's width alone, so lengths are taken to be as long as that: a
    // table of 128 pages of 64 for the same sequence has its units cut (64 / 256 tokens: 8.4 /
    // 11.0 us against 6.1 / 8.3 with tables of 1 and 4 pages).
    // 4-bit rows take longer to expand than to read: two granules (d = 128, 256 tokens: 8.8
    // us against 9.9; d = 512, 256 tokens: 17.0 against 17.7)
    const bool whole = units <= grid && (INT4 ? granules <= 2 : keys * 4 * D <= 160 * 1024);
    fa::PagedFwdParams a = p;
    a.coarse = whole ? static_cast<int>(granules) : 1;
    if (whole) a.rec = nullptr;
    const double most = whole ? units : units * granules;
    if (most < grid) grid = static_cast<int>(most);
    kernel<<<grid, C::THREADS, C::SMEM, s>>>(a);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    if (whole) return FA_OK;
    // the join starts its blocks while the forward's last CTAs run, and waits for them
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    // a block per cut unit; where pieces per unit are many, or blocks few, a block per row
    // of it (one sequence of 1000 tokens, 8 KV heads: 9.3 us in all against 13.3; 64
    // sequences up to 8192 tokens, 4 KV heads: 94.7 us with a block per row, 93.9 with one)
    cfg.gridDim = dim3(grid, units * 8 < grid || grid * C::ROWS <= 1024 ? C::ROWS : 1);
    cfg.blockDim = dim3(fa::kJoinWarps * 32);
    cfg.stream = s;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fa::fa_fwd_paged_join_kernel<D, BF16, C::ROWS>, a) == cudaSuccess ? FA_OK
                                                                                                           : FA_ERR_CUDA;
}

template <int D, int NT>
fa_status launch_paged_types(const fa::PagedFwdParams& p, bool bf16, bool int4, int sm_count, cudaStream_t s)
{
    if (int4) return bf16 ? launch_paged<D, true, true, NT>(p, sm_count, s) : launch_paged<D, false, true, NT>(p, sm_count, s);
    return bf16 ? launch_paged<D, true, false, NT>(p, sm_count, s) : launch_paged<D, false, false, NT>(p, sm_count, s);
}

template <int D>
fa_status launch_paged_rows(const fa::PagedFwdParams& p, int nt, bool bf16, bool int4, int sm_count, cudaStream_t s)
{
    if constexpr (D == 128)
        if (nt == 4) return launch_paged_types<D, 4>(p, bf16, int4, sm_count, s);
    if constexpr (D <= 256)
        if (nt == 2) return launch_paged_types<D, 2>(p, bf16, int4, sm_count, s);
    return launch_paged_types<D, 1>(p, bf16, int4, sm_count, s);
}

}  // namespace

extern "C" {

size_t fa_kv_cache_size(int num_pages, int page_size, int Hkv, int d, fa_kv_format fmt)
{
    if (num_pages < 1 || !page_size_ok(page_size) || Hkv < 1 || !head_dim_ok(d) ||
        (fmt != FA_KV_16 && fmt != FA_KV_INT4))
        return 0;
    return static_cast<size_t>(num_pages) * Hkv * page_size * (fmt == FA_KV_16 ? 2 * d : 5 * d / 8);
}

fa_status fa_kv_append(const void* q, const void* k, const void* v, long long q_stride, long long k_stride,
                       long long v_stride, void* q_out, void* k_cache, void* v_cache, const int* cu_seqlens,
                       const int* seqlens_k, const int* block_table, const float* inv_freq, int rot_dim,
                       int interleaved, int B, int total, int Hq, int Hkv, int d, int page_size, int num_pages,
                       int max_pages, fa_kv_format fmt, fa_dtype dt, fa_stream stream)
{
    fa::AppendParams p{};
    fa_status st = check_pool(k_cache, v_cache, block_table, B, Hkv, d, page_size, num_pages, max_pages, fmt, dt,
                              &p.pool);
    if (st != FA_OK) return st;
    if (!cu_seqlens || !seqlens_k || !aligned4(cu_seqlens) || !aligned4(seqlens_k)) return FA_ERR_INVALID_ARG;
    if (total < 0 || Hq < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
    if (rot_dim < 0 || rot_dim > d || rot_dim % 16 != 0) return FA_ERR_INVALID_ARG;
    if (rot_dim > 0 && (!inv_freq || !aligned4(inv_freq))) return FA_ERR_INVALID_ARG;
    if (total == 0) return FA_OK;
    if (!k || !v || (q == nullptr) != (q_out == nullptr)) return FA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out)) return FA_ERR_INVALID_ARG;
    if (q && (q_stride % 8 != 0 || q_stride < static_cast<long long>(Hq) * d)) return FA_ERR_INVALID_ARG;
    if (q && q == q_out && q_stride != static_cast<long long>(Hq) * d) return FA_ERR_INVALID_ARG;
    if (k_stride % 8 != 0 || v_stride % 8 != 0 || k_stride < static_cast<long long>(Hkv) * d ||
        v_stride < static_cast<long long>(Hkv) * d)
        return FA_ERR_INVALID_ARG;
    // a block's items are counted in 32 bits
    if (static_cast<long long>(Hq) * d >= (1LL << 24)) return FA_ERR_INVALID_ARG;
    DeviceInfo di;
    st = device_info(&di);
    if (st != FA_OK) return st;
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.q_out = q_out;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.cu = cu_seqlens;
    p.seqlens_k = seqlens_k;
    p.inv_freq = inv_freq;
    p.rot = rot_dim;
    p.interleaved = interleaved ? 1 : 0;
    p.B = B;
    p.total = total;
    p.Hq = Hq;
    p.tpb = total >= 8 * di.sm_count ? fa::kAppendTokens : 1;
    const unsigned blocks = (static_cast<unsigned>(total) + p.tpb - 1) / p.tpb;
    const bool bf16 = dt == FA_BF16, int4 = fmt == FA_KV_INT4;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (d) {
    case 128: return launch_append<128>(p, blocks, bf16, int4, s);
    case 192: return launch_append<192>(p, blocks, bf16, int4, s);
    case 256: return launch_append<256>(p, blocks, bf16, int4, s);
    case 384: return launch_append<384>(p, blocks, bf16, int4, s);
    default: return launch_append<512>(p, blocks, bf16, int4, s);
    }
}

fa_status fa_kv_gather(const void* k_cache, const void* v_cache, void* k, void* v, const int* cu_seqlens_k,
                       const int* block_table, int B, int total_k, int Hkv, int d, int page_size, int num_pages,
                       int max_pages, fa_kv_format fmt, fa_dtype dt, fa_stream stream)
{
    fa::GatherParams p{};
    fa_status st = check_pool(k_cache, v_cache, block_table, B, Hkv, d, page_size, num_pages, max_pages, fmt, dt,
                              &p.pool);
    if (st != FA_OK) return st;
    if (!cu_seqlens_k || !aligned4(cu_seqlens_k) || total_k < 0) return FA_ERR_INVALID_ARG;
    if (total_k == 0) return FA_OK;
    if (!k || !v || !aligned16(k) || !aligned16(v)) return FA_ERR_INVALID_ARG;
    if (static_cast<long long>(Hkv) * d >= (1LL << 24)) return FA_ERR_INVALID_ARG;
    DeviceInfo di;
    st = device_info(&di);
    if (st != FA_OK) return st;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.k = k;
    p.v = v;
    p.cu = cu_seqlens_k;
    p.B = B;
    p.total = total_k;
    const unsigned blocks = (static_cast<unsigned>(total_k) + fa::kGatherTokens - 1) / fa::kGatherTokens;
    const bool bf16 = dt == FA_BF16, int4 = fmt == FA_KV_INT4;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (d) {
    case 128: return launch_gather<128>(p, blocks, bf16, int4, s);
    case 192: return launch_gather<192>(p, blocks, bf16, int4, s);
    case 256: return launch_gather<256>(p, blocks, bf16, int4, s);
    case 384: return launch_gather<384>(p, blocks, bf16, int4, s);
    default: return launch_gather<512>(p, blocks, bf16, int4, s);
    }
}

size_t fa_fwd_paged_workspace_size(int B, int max_seqlen_q, int Hq, int Hkv, int d)
{
    if (B < 1 || max_seqlen_q < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || !head_dim_ok(d)) return 0;
    DeviceInfo di;
    if (device_info(&di) != FA_OK) return 0;
    return paged_workspace(di.sm_count, 8 * paged_tiles(max_seqlen_q, Hq / Hkv, d), d, nullptr, nullptr);
}

fa_status fa_fwd_paged(const void* q, const void* k_cache, const void* v_cache, void* o, float* lse,
                       const int* cu_seqlens_q, const int* seqlens_k, const int* block_table, int B,
                       int max_seqlen_q, int total_q, int Hq, int Hkv, int d, int page_size, int num_pages,
                       int max_pages, fa_kv_format fmt, int causal, float scale, fa_dtype dt, void* workspace,
                       size_t workspace_bytes, fa_stream stream)
{
    fa::PagedFwdParams p{};
    fa_status st = check_pool(k_cache, v_cache, block_table, B, Hkv, d, page_size, num_pages, max_pages, fmt, dt,
                              &p.pool);
    if (st != FA_OK) return st;
    if (!cu_seqlens_q || !seqlens_k || !aligned4(cu_seqlens_q) || !aligned4(seqlens_k)) return FA_ERR_INVALID_ARG;
    if (max_seqlen_q < 1 || total_q < 0 || Hq < 1 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.0f)) return FA_ERR_INVALID_ARG;
    if (static_cast<long long>(total_q) * Hq >= (1LL << 31)) return FA_ERR_INVALID_ARG;
    if (total_q == 0) return FA_OK;
    if (!q || !o || !lse || !aligned16(q) || !aligned16(o) || !aligned16(lse)) return FA_ERR_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u)) return FA_ERR_INVALID_ARG;
    DeviceInfo di;
    st = device_info(&di);
    if (st != FA_OK) return st;
    const int nt = paged_tiles(max_seqlen_q, Hq / Hkv, d);
    if (workspace_bytes < paged_workspace(di.sm_count, 8 * nt, d, &p, workspace)) return FA_ERR_INVALID_ARG;
    p.q = q;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.o = o;
    p.lse = lse;
    p.cu_q = cu_seqlens_q;
    p.seqlens_k = seqlens_k;
    p.B = B;
    p.max_q = max_seqlen_q;
    p.total_q = total_q;
    p.Hq = Hq;
    p.group = Hq / Hkv;
    p.by_group = fa::Divider::by(p.group);
    p.by_hkv = fa::Divider::by(Hkv);
    p.causal = causal ? 1 : 0;
    p.sl2 = scale * 1.4426950408889634f;
    const bool bf16 = dt == FA_BF16, int4 = fmt == FA_KV_INT4;
    p.block_bytes = static_cast<uint32_t>(page_size) * (int4 ? 5 * d / 8 : 2 * d);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    switch (d) {
    case 128: return launch_paged_rows<128>(p, nt, bf16, int4, di.sm_count, s);
    case 192: return launch_paged_rows<192>(p, nt, bf16, int4, di.sm_count, s);
    case 256: return launch_paged_rows<256>(p, nt, bf16, int4, di.sm_count, s);
    case 384: return launch_paged_rows<384>(p, nt, bf16, int4, di.sm_count, s);
    default: return launch_paged_rows<512>(p, nt, bf16, int4, di.sm_count, s);
    }
}

}  // extern "C"
