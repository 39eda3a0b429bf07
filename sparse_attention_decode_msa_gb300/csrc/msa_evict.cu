// msa_evict.cu -- eviction of cached positions by accumulated weight
// (msa_cache_evict): which positions stay, and their rows copied to new pages.
//
// A list keeps `keep` of the n cached positions: the first `first` and the
// last `last`, then the largest weights, ties to the lower position; it is
// ascending, so the shortened cache holds its tokens in their old order.  With
// one index head there is one list a request, on the maximum over KV heads of
// their weights (a maximum, not a sum: exact whatever the order of the heads,
// as the block select's reduction is); with more, one list per KV head.
//
// Select: comparisons only, so bit-exact.  A cluster of 8 CTAs per list, each
// with an eighth of the positions, whose order-preserving 32-bit keys stay in
// shared memory (up to 40960 a CTA; longer slices read the weights again).
// Three digits (11, 11, 10 bits) from the top give the keep-th largest key:
// histograms are summed over the cluster through distributed shared memory.
// Prefix counts in position order then give each kept position its place.
//
// Copy: 64 kept positions per CTA; every row is 16-byte pieces, several loads
// in flight per thread.  Rows go to pages of their own (new_table), so pages
// that other requests share stay as they are and no copy waits for another.
#include "msa_cache.cuh"

namespace msa {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kCluster = 8;
constexpr int kKeysHeld = 40960;
constexpr int kBins = 2048;

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A 32-bit word of another CTA's shared memory.
__device__ __forceinline__ int ld_peer(const void *p, int rank)
{
    uint32_t a;
    int v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

// Exclusive scan over the CTA; *total gets the sum.  tmp: kSelWarps + 1 words.
__device__ __forceinline__ uint32_t cta_scan(uint32_t v, uint32_t *tmp, uint32_t *total)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += u;
    }
    if (lane == 31)
        tmp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        const uint32_t w = lane < kSelWarps ? tmp[lane] : 0u;
        uint32_t wi = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, wi, o);
            if (lane >= o)
                wi += u;
        }
        if (lane < kSelWarps)
            tmp[lane] = wi - w;
        if (lane == kSelWarps - 1)
            tmp[kSelWarps] = wi;
    }
    __syncthreads();
    const uint32_t res = tmp[warp] + incl - v;
    *total = tmp[kSelWarps];
    __syncthreads();
    return res;
}

// Key of one weight; NaN ranks above every number, below the forced positions.
__device__ __forceinline__ uint32_t weight_key(float w)
{
    return w != w ? 0xFFFFFFFEu : order_key(w);
}

// Key of position `at`: w points at the list's first KV head, `heads` rows of `pitch`.
__device__ __forceinline__ uint32_t position_key(const EvictParams &p, const float *w, int heads, size_t pitch, int at, int n)
{
    if (at < p.first || at >= n - p.last)
        return 0xFFFFFFFFu;
    uint32_t k = 0u;
    for (int h = 0; h < heads; ++h)
        k = max(k, weight_key(w[h * pitch + at]));
    return k;
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p, int held)
{
    extern __shared__ uint32_t keys[]; // [held]
    __shared__ int hist[2][kBins];
    __shared__ uint32_t scan_tmp[kSelWarps + 1];
    __shared__ int s_digit, s_need, s_counts[2];

    launch_dependents();
    const int list = blockIdx.x / kCluster, rank = (int)cluster_rank();
    const int r = list / p.Hs, hs = list - r * p.Hs;
    const int heads = p.Hkv / p.Hs;
    int32_t *out = p.kept + (size_t)list * p.keep;
    const int seq_len = p.seq_lens[r];
    bool bad;
    const int nb = cached_blocks(seq_len, p.nq, p.maxB, &bad);
    if (bad && rank == 0 && threadIdx.x == 0)
        set_error(p.err, kErrSeqLen);
    const int n = nb == 0 ? 0 : seq_len + p.nq - 1;
    if (hs == 0 && rank == 0 && threadIdx.x == 0)
        p.new_lens[r] = n == 0 ? 0 : min(n, p.keep) - p.nq + 1;
    if (n <= p.keep) { // everything stays (the whole cluster takes this branch)
        for (int i = rank * kSelThreads + threadIdx.x; i < p.keep; i += kCluster * kSelThreads)
            out[i] = i < n ? i : -1;
        return;
    }

    const int slice = ((n + kCluster - 1) / kCluster + 3) & ~3;
    const int lo = min(n, rank * slice), hi = min(n, lo + slice), count = hi - lo;
    const size_t pitch = (size_t)p.maxB * kPage;
    const float *w = p.weights + ((size_t)r * p.Hkv + (size_t)hs * heads) * pitch;
    const bool cached = count <= held;
    if (cached)
        for (int i = threadIdx.x; i < count; i += kSelThreads)
            keys[i] = position_key(p, w, heads, pitch, lo + i, n);
    auto key = [&](int i) { return cached ? keys[i] : position_key(p, w, heads, pitch, lo + i, n); };

    // the keep-th largest key, digit by digit
    uint32_t prefix = 0u;
    int need = p.keep;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        int *h = hist[pass & 1];
        for (int i = threadIdx.x; i < kBins; i += kSelThreads)
            h[i] = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < count; i += kSelThreads) {
            const uint32_t k = key(i);
            if (pass == 0 || (k >> (shift + bits)) == prefix)
                atomicAdd(&h[(k >> shift) & ((1u << bits) - 1u)], 1);
        }
        cluster_sync();
        // bins from the top: thread t has the 4 bins kBins - 1 - 4 t and below
        int c[4];
        uint32_t sum = 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            c[k] = 0;
            for (int q = 0; q < kCluster; ++q)
                c[k] += ld_peer(&h[kBins - 1 - 4 * (int)threadIdx.x - k], q);
            sum += (uint32_t)c[k];
        }
        uint32_t total;
        int above = (int)cta_scan(sum, scan_tmp, &total);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (above < need && need <= above + c[k]) { // one bin of one thread
                s_digit = kBins - 1 - 4 * (int)threadIdx.x - k;
                s_need = need - above;
            }
            above += c[k];
        }
        __syncthreads();
        prefix = (prefix << bits) | (uint32_t)s_digit;
        need = s_need;
        __syncthreads();
    }
    const uint32_t theta = prefix; // kept: keys above theta, and the first `need` equal to it

    int gt = 0, eq = 0;
    for (int i = threadIdx.x; i < count; i += kSelThreads) {
        const uint32_t k = key(i);
        gt += k > theta;
        eq += k == theta;
    }
    uint32_t total_gt, total_eq;
    cta_scan((uint32_t)gt, scan_tmp, &total_gt);
    cta_scan((uint32_t)eq, scan_tmp, &total_eq);
    if (threadIdx.x == 0) {
        s_counts[0] = (int)total_gt;
        s_counts[1] = (int)total_eq;
    }
    cluster_sync();
    int gt_before = 0, eq_before = 0;
    for (int q = 0; q < rank; ++q) {
        gt_before += ld_peer(&s_counts[0], q);
        eq_before += ld_peer(&s_counts[1], q);
    }
    cluster_sync(); // no CTA leaves while another reads its counts

    for (int i0 = 0; i0 < count; i0 += kSelThreads * 4) {
        const int i = i0 + 4 * (int)threadIdx.x;
        uint32_t k[4];
        uint32_t mine = 0u; // at most 2048 of each kind: two 16-bit counts
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            k[e] = i + e < count ? key(i + e) : 0u;
            const bool in = i + e < count;
            mine += (in && k[e] > theta ? 1u : 0u) + (in && k[e] == theta ? 0x10000u : 0u);
        }
        uint32_t total;
        const uint32_t before = cta_scan(mine, scan_tmp, &total);
        int g = gt_before + (int)(before & 0xFFFFu), q = eq_before + (int)(before >> 16);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (i + e >= count)
                break;
            const bool is_gt = k[e] > theta, is_eq = k[e] == theta;
            if (is_gt || (is_eq && q < need))
                out[g + min(q, need)] = lo + i + e;
            g += is_gt;
            q += is_eq;
        }
        gt_before += (int)(total & 0xFFFFu);
        eq_before += (int)(total >> 16);
    }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyRows = 64; // kept positions of a CTA

// Copies `kinds` rows of PIECES pieces of type T for each of the CTA's `count`
// positions: piece i of kind k from src row to dst row, at `base(k, page) + row * pitch`.
template <typename T, typename F>
__device__ __forceinline__ void copy_rows(int kinds, int pieces, int count, const int2 *from, const int2 *to, F &&at)
{
    const int total = kinds * kCopyRows * pieces;
    constexpr int U = 8; // loads in flight
    for (int i0 = threadIdx.x; i0 < total; i0 += U * kCopyThreads) {
        T v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kCopyThreads, e = (i / pieces) % kCopyRows;
            if (i < total && e < count && from[e].x >= 0 && to[e].x >= 0)
                v[u] = *reinterpret_cast<const T *>(at(i / (pieces * kCopyRows), from[e], i % pieces));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * kCopyThreads, e = (i / pieces) % kCopyRows;
            if (i < total && e < count && from[e].x >= 0 && to[e].x >= 0)
                *reinterpret_cast<T *>(at(i / (pieces * kCopyRows), to[e], i % pieces)) = v[u];
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictParams p)
{
    __shared__ int2 from[kCopyRows], to[kCopyRows]; // page, row of the page; page -1: not copied
    __shared__ int pos[kCopyRows];
    const int list = blockIdx.x, r = list / p.Hs, hs = list - r * p.Hs;
    const int heads = p.Hkv / p.Hs, index_heads = p.Hi / p.Hs;
    const int i0 = blockIdx.y * kCopyRows;
    grid_dependency_wait();
    if (threadIdx.x < kCopyRows) {
        const int i = i0 + threadIdx.x;
        int2 f = make_int2(-1, 0), t = make_int2(-1, 0);
        int at = -1;
        if (i < p.keep)
            at = p.kept[(size_t)list * p.keep + i];
        if (at >= 0) {
            f = make_int2(p.block_table[(size_t)r * p.maxB + at / kPage], at % kPage);
            t = make_int2(p.new_table[(size_t)r * p.newB + i / kPage], i % kPage);
            if (f.x < 0 || f.x >= p.num_pages || t.x < 0 || t.x >= p.num_pages) {
                set_error(p.err, kErrPage);
                f.x = t.x = -1;
            }
        }
        from[threadIdx.x] = f;
        to[threadIdx.x] = t;
        pos[threadIdx.x] = at;
    }
    __syncthreads();
    const int count = min(kCopyRows, p.keep - i0);
    if (pos[0] < 0)
        return; // the lists are filled from the front

    // K rows of the list's KV heads, then V rows
    const int fmt = p.kv_fmt;
    auto tile = [&](int k, int page) { // kind k: K of head k, then V
        const int v = k >= heads, g = hs * heads + (v ? k - heads : k);
        return ((size_t)page * 2 + v) * p.Hkv + g;
    };
    if (fmt == kFmtF4) {
        copy_rows<uint4>(2 * heads, 4, count, from, to, [&](int k, int2 a, int i) {
            return p.kv + tile(k, a.x) * 9216 + a.y * 64 + i * 16;
        });
        copy_rows<uint2>(2 * heads, 1, count, from, to, [&](int k, int2 a, int) {
            return p.kv + tile(k, a.x) * 9216 + 8192 + a.y * 8;
        });
    } else {
        const int row_bytes = fmt == kFmtBf16 ? 256 : 128;
        copy_rows<uint4>(2 * heads, row_bytes / 16, count, from, to, [&](int k, int2 a, int i) {
            return p.kv + (tile(k, a.x) * kPage + a.y) * row_bytes + i * 16;
        });
    }
    if (p.idxk) {
        auto row = [&](int k, int2 a) { return ((size_t)a.x * p.Hi + hs * index_heads + k) * kPage + a.y; };
        const int row_bytes = p.idx_f4 ? 64 : 256;
        copy_rows<uint4>(index_heads, row_bytes / 16, count, from, to, [&](int k, int2 a, int i) {
            return p.idxk + row(k, a) * row_bytes + i * 16;
        });
        if (p.idx_f4)
            copy_rows<uint2>(index_heads, 1, count, from, to, [&](int k, int2 a, int) { return p.idxk_scales + row(k, a) * 8; });
    }
    if (p.new_weights)
        for (int i = threadIdx.x; i < heads * kCopyRows; i += kCopyThreads) {
            const int e = i % kCopyRows, g = hs * heads + i / kCopyRows;
            if (e < count && pos[e] >= 0)
                p.new_weights[((size_t)r * p.Hkv + g) * p.newB * kPage + i0 + e] =
                    p.weights[((size_t)r * p.Hkv + g) * p.maxB * kPage + pos[e]];
        }
}

} // namespace

cudaError_t launch_cache_evict(const EvictParams &p, cudaStream_t stream)
{
    const int lists = p.R * p.Hs;
    // keys of a slice of the longest row the table can hold, as far as they are held
    const long long slice = ((long long)p.maxB * kPage + kCluster - 1) / kCluster + 3;
    const int held = slice < kKeysHeld ? (int)slice : kKeysHeld;
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysHeld * 4);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(lists * kCluster);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (size_t)held * 4;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, held);
    if (e == cudaSuccess)
        e = launch_kernel(evict_copy_kernel, dim3(lists, (p.keep + kCopyRows - 1) / kCopyRows), dim3(kCopyThreads), 0, stream, true, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace msa
