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
// Select: comparisons only, so bit-exact.  One CTA per list where the table
// holds at most 8192 positions, else a cluster of 8 (a whole eviction of 8 x 2048
// positions 13.9 us, 17.5 with clusters; of 2 x 4096 14.7 and 14.5; of 8 x 32768
// 74 us with one CTA a list, 47 with clusters), each CTA with an eighth of the positions, whose order-preserving 32-bit keys stay in shared memory (up to
// 40960 a CTA; longer slices read the weights again).  Four 8-bit digits from the
// top give the keep-th largest key: the CTAs read one another's histograms (256
// words; with 11-bit digits their reading took as long as all the rest of a digit)
// through distributed shared memory, one cluster barrier a digit, and from the same
// words how many kept positions the CTAs before them have.  Eight copies of the
// histogram, by lane, keep a warp's increments of one word apart.  Prefix counts in
// position order then give each kept position its place.
//
// Copy: 128 kept positions per CTA, or 32 where that leaves fewer CTAs than two per SM
// (1024 positions cut to 512: 10.2 us for 15.6; 32 lists of 65536 positions: 168 us with
// 32, 123 with 128); every row is 16-byte pieces, eight loads in flight per thread over
// K, V and index-key rows alike.  Rows go to pages of their own (new_table), so pages
// that other requests share stay as they are and no copy waits for another.
//
// What bounds it: HBM for long lists (268 MB of rows read and written in 94 us, 5.7 TB/s), the
// chain of four digits before the copy (29 of 123 us), launch latency for short ones.
#include "msa_cache.cuh"

namespace msa {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kCluster = 8;
constexpr int kKeysHeld = 40960;
constexpr int kBins = 256;
constexpr int kCopies = 8;

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

template <int CLUSTER>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p, int held)
{
    extern __shared__ __align__(16) uint32_t keys[]; // [held]
    __shared__ int copies[kCopies][kBins], hist[4][kBins];
    __shared__ uint32_t scan_tmp[kSelWarps + 1];
    __shared__ int s_digit, s_need, s_before, s_equal;

    launch_dependents();
    const int list = blockIdx.x / CLUSTER, rank = CLUSTER > 1 ? (int)cluster_rank() : 0;
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
        for (int i = rank * kSelThreads + threadIdx.x; i < p.keep; i += CLUSTER * kSelThreads)
            out[i] = i < n ? i : -1;
        return;
    }

    const int slice = ((n + CLUSTER - 1) / CLUSTER + 3) & ~3;
    const int lo = min(n, rank * slice), hi = min(n, lo + slice), count = hi - lo;
    const size_t pitch = (size_t)p.maxB * kPage;
    const float *w = p.weights + ((size_t)r * p.Hkv + (size_t)hs * heads) * pitch;
    const bool cached = count <= held;
    for (int i = threadIdx.x; i < kCopies * kBins; i += kSelThreads)
        (&copies[0][0])[i] = 0;
    if (threadIdx.x == 0)
        s_before = 0;
    __syncthreads();
    auto key = [&](int i) { return cached ? keys[i] : position_key(p, w, heads, pitch, lo + i, n); };
    // keys four at a time (rows are multiples of 128 long), the first digit counted as they come
    auto four_keys = [&](int i, uint32_t (&k)[4]) {
        k[0] = k[1] = k[2] = k[3] = 0u;
        for (int h = 0; h < heads; ++h) {
            const float4 v = *reinterpret_cast<const float4 *>(w + h * pitch + lo + i);
            k[0] = max(k[0], weight_key(v.x));
            k[1] = max(k[1], weight_key(v.y));
            k[2] = max(k[2], weight_key(v.z));
            k[3] = max(k[3], weight_key(v.w));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (lo + i + e < p.first || lo + i + e >= n - p.last)
                k[e] = 0xFFFFFFFFu;
    };
    constexpr int U = 4; // loads in flight a thread
    int *mine = copies[threadIdx.x & (kCopies - 1)];
    for (int i0 = 4 * (int)threadIdx.x; i0 < count; i0 += 4 * U * kSelThreads) {
        uint32_t k[U][4];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (i0 + 4 * u * kSelThreads < count)
                four_keys(i0 + 4 * u * kSelThreads, k[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + 4 * u * kSelThreads;
            if (i >= count)
                break;
            if (cached)
                *reinterpret_cast<uint4 *>(keys + i) = make_uint4(k[u][0], k[u][1], k[u][2], k[u][3]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < count)
                    atomicAdd(&mine[k[u][e] >> 24], 1);
        }
    }
    // the keep-th largest key, digit by digit
    uint32_t prefix = 0u;
    int need = p.keep;
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        if (pass > 0) {
            auto add = [&](uint32_t k) {
                if ((k >> (shift + 8)) == prefix)
                    atomicAdd(&mine[(k >> shift) & 255u], 1);
            };
            const int whole = cached ? count & ~3 : 0;
            for (int i = 4 * (int)threadIdx.x; i < whole; i += 4 * kSelThreads) {
                const uint4 k = *reinterpret_cast<const uint4 *>(keys + i);
                add(k.x);
                add(k.y);
                add(k.z);
                add(k.w);
            }
            for (int i = whole + threadIdx.x; i < count; i += kSelThreads)
                add(key(i));
        }
        __syncthreads();
        if (threadIdx.x < kBins) {
            int sum = 0;
#pragma unroll
            for (int c = 0; c < kCopies; ++c) {
                sum += copies[c][threadIdx.x];
                copies[c][threadIdx.x] = 0;
            }
            hist[pass][threadIdx.x] = sum;
        }
        if (CLUSTER > 1)
            cluster_sync();
        else
            __syncthreads();
        // thread t has bin kBins - 1 - t: of all CTAs, and of those before this one
        const int bin = kBins - 1 - (int)threadIdx.x;
        int c = 0, before = 0;
        if (bin >= 0) {
            int v[CLUSTER];
#pragma unroll
            for (int q = 0; q < CLUSTER; ++q)
                v[q] = CLUSTER > 1 ? ld_peer(&hist[pass][bin], q) : hist[pass][bin];
#pragma unroll
            for (int q = 0; q < CLUSTER; ++q) {
                c += v[q];
                before += q < rank ? v[q] : 0;
            }
        }
        uint32_t total;
        const int above = (int)cta_scan((uint32_t)c, scan_tmp, &total);
        if (above < need && need <= above + c) { // one bin
            s_digit = bin;
            s_need = need - above;
            s_equal = before;
        }
        __syncthreads();
        // positions of the CTAs before this one that are kept by this digit
        const int kept = (int)__reduce_add_sync(0xffffffffu, bin > s_digit ? (uint32_t)before : 0u);
        if ((threadIdx.x & 31) == 0 && kept)
            atomicAdd(&s_before, kept);
        prefix = (prefix << 8) | (uint32_t)s_digit;
        need = s_need;
        __syncthreads();
    }
    const uint32_t theta = prefix; // kept: keys above theta, and the first `need` equal to it
    const int gt_before = s_before, eq_before = s_equal;
    if (CLUSTER > 1) // no CTA leaves while another reads its histograms
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

    // every thread has a run of consecutive positions, an odd number of 16-byte words of
    // keys (no bank conflicts): one scan over the CTA places all of them
    const int run = ((((count + kSelThreads - 1) / kSelThreads + 3) >> 2) | 1) << 2;
    const int begin = min(count, run * (int)threadIdx.x), end = min(count, begin + run);
    auto four = [&](int i, uint32_t (&k)[4]) { // of this thread's run
        if (cached) {
            const uint4 v = *reinterpret_cast<const uint4 *>(keys + i);
            k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                k[e] = i + e < end ? key(i + e) : 0u;
        }
    };
    int gt = 0, eq = 0;
    for (int i = begin; i < end; i += 4) {
        uint32_t k[4];
        four(i, k);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            gt += i + e < end && k[e] > theta;
            eq += i + e < end && k[e] == theta;
        }
    }
    uint32_t total;
    int g = gt_before + (int)cta_scan((uint32_t)gt, scan_tmp, &total);
    int q = eq_before + (int)cta_scan((uint32_t)eq, scan_tmp, &total);
    if (gt || (eq && q < need))
        for (int i = begin; i < end; i += 4) {
            uint32_t k[4];
            four(i, k);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const bool is_gt = i + e < end && k[e] > theta, is_eq = i + e < end && k[e] == theta;
                if (is_gt || (is_eq && q < need))
                    out[g + min(q, need)] = lo + i + e;
                g += is_gt;
                q += is_eq;
            }
        }
    if (CLUSTER > 1)
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kCopyThreads = 256;

__device__ __forceinline__ int log2_of(int v) // of a power of two
{
    return 31 - __clz(v);
}

// ROWS kept positions of one list.
template <int ROWS>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictParams p)
{
    __shared__ int2 from[ROWS], to[ROWS]; // page, row of the page; page -1: not copied
    __shared__ int pos[ROWS];
    const int list = blockIdx.x, r = list / p.Hs, hs = list - r * p.Hs;
    const int heads = p.Hkv / p.Hs, index_heads = p.idxk ? p.Hi / p.Hs : 0;
    const int i0 = blockIdx.y * ROWS;
    grid_dependency_wait();
    if (threadIdx.x < ROWS) {
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
    if (pos[0] < 0)
        return; // the lists are filled from the front

    // rows in 16-byte pieces: K of the list's KV heads, V of them, then their index keys.
    // NVFP4 rows are 64 bytes of codes here and 8 of scales below.
    const bool f4 = p.kv_fmt == kFmtF4;
    const int kv_row = f4 ? 64 : p.kv_fmt == kFmtFp8 ? 128 : 256, idx_row = p.idx_f4 ? 64 : 256;
    const int kv_shift = log2_of(kv_row >> 4), idx_shift = log2_of(idx_row >> 4), kv_page = f4 ? 9216 : kPage * kv_row;
    auto tile = [&](int k, int page) { // kind k: K of head k, then V
        const int v = k >= heads, g = hs * heads + (v ? k - heads : k);
        return ((size_t)page * 2 + v) * p.Hkv + g;
    };
    const int kv_pieces = 2 * heads * ROWS << kv_shift, pieces = kv_pieces + (index_heads * ROWS << idx_shift);
    auto row_of = [&](int i) { return (i < kv_pieces ? i >> kv_shift : (i - kv_pieces) >> idx_shift) & (ROWS - 1); };
    auto piece_at = [&](int i, int2 a) -> uint4 * {
        if (i < kv_pieces)
            return reinterpret_cast<uint4 *>(p.kv + tile(i >> kv_shift >> log2_of(ROWS), a.x) * kv_page + a.y * kv_row) + (i & ((1 << kv_shift) - 1));
        i -= kv_pieces;
        const size_t h = (size_t)a.x * p.Hi + hs * index_heads + (i >> idx_shift >> log2_of(ROWS));
        return reinterpret_cast<uint4 *>(p.idxk + (h * kPage + a.y) * idx_row) + (i & ((1 << idx_shift) - 1));
    };
    constexpr int U = 8; // loads in flight
    for (int j0 = threadIdx.x; j0 < pieces; j0 += U * kCopyThreads) {
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = j0 + u * kCopyThreads;
            if (i < pieces && from[row_of(i)].x >= 0)
                v[u] = *piece_at(i, from[row_of(i)]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = j0 + u * kCopyThreads;
            if (i < pieces && from[row_of(i)].x >= 0)
                *piece_at(i, to[row_of(i)]) = v[u];
        }
    }
    if (f4) // 8 scales a row
        for (int i = threadIdx.x; i < 2 * heads * ROWS; i += kCopyThreads) {
            const int2 a = from[i % ROWS], b = to[i % ROWS];
            if (a.x >= 0)
                *reinterpret_cast<uint2 *>(p.kv + tile(i / ROWS, b.x) * 9216 + 8192 + b.y * 8) =
                    *reinterpret_cast<const uint2 *>(p.kv + tile(i / ROWS, a.x) * 9216 + 8192 + a.y * 8);
        }
    if (p.idx_f4)
        for (int i = threadIdx.x; i < index_heads * ROWS; i += kCopyThreads) {
            const int2 a = from[i % ROWS], b = to[i % ROWS];
            const int h = hs * index_heads + i / ROWS;
            if (a.x >= 0)
                *reinterpret_cast<uint2 *>(p.idxk_scales + (((size_t)b.x * p.Hi + h) * kPage + b.y) * 8) =
                    *reinterpret_cast<const uint2 *>(p.idxk_scales + (((size_t)a.x * p.Hi + h) * kPage + a.y) * 8);
        }
    if (p.new_weights)
        for (int i = threadIdx.x; i < heads * ROWS; i += kCopyThreads) {
            const int e = i % ROWS, g = hs * heads + i / ROWS;
            if (pos[e] >= 0)
                p.new_weights[((size_t)r * p.Hkv + g) * p.newB * kPage + i0 + e] =
                    p.weights[((size_t)r * p.Hkv + g) * p.maxB * kPage + pos[e]];
        }
}

template <int CLUSTER>
cudaError_t launch_select_t(const EvictParams &p, cudaStream_t stream)
{
    const int lists = p.R * p.Hs;
    // keys of a slice of the longest row the table can hold, as far as they are held
    const long long slice = ((long long)p.maxB * kPage + CLUSTER - 1) / CLUSTER + 4;
    const int held = slice < kKeysHeld ? (int)slice : kKeysHeld;
    cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<CLUSTER>, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysHeld * 4);
    if (e != cudaSuccess)
        return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CLUSTER;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(lists * CLUSTER);
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = (size_t)held * 4;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = CLUSTER > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<CLUSTER>, p, held);
}

} // namespace

cudaError_t launch_cache_evict(const EvictParams &p, cudaStream_t stream)
{
    cudaError_t e = p.maxB * kPage <= 8192 ? launch_select_t<1>(p, stream) : launch_select_t<kCluster>(p, stream);
    if (e != cudaSuccess)
        return e;
    // short lists in more, smaller CTAs (both measured: see the top)
    const int lists = p.R * p.Hs;
    if ((long long)lists * ((p.keep + 127) / 128) >= 304)
        e = launch_kernel(evict_copy_kernel<128>, dim3(lists, (p.keep + 127) / 128), dim3(kCopyThreads), 0, stream, true, p);
    else
        e = launch_kernel(evict_copy_kernel<32>, dim3(lists, (p.keep + 31) / 32), dim3(kCopyThreads), 0, stream, true, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

} // namespace msa
