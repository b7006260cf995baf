// kv_pages.cu -- the pages of the attention cache: rows resized (with copy on write), forked and compacted, and
// the data copied.
//
// Whole numbers only: a page's count of holders, rows of page indices, lengths.  The allocation order is defined
// (lowest free page first, lanes in order), so results do not depend on timing: what runs in any order is counts
// that are added to.  Resizing and compacting need the free pages in order, a scan over all counts: a cluster of
// CTAs takes equal parts of them and passes the parts' numbers through distributed shared memory, in one launch.
//
// Copies are HBM-bound, the rest is latency: 64 prompts of up to 3,000 tokens forked eight times each and grown by a token, with
// the 512 copies of shared last pages (134 MB read and written, 8 samples from one source) 52 us; 31 us for five samples of one
// prompt, four calls of about 4 us on the GPU that the host takes 7 us each to issue; a compaction that moves 0.5 GB 175 us, 0.87
// of the copy rate.
#include <cooperative_groups.h>

#include "attn_common.cuh"

namespace cg = cooperative_groups;

namespace gdn {

namespace {

constexpr int kPageThreads = 1024;
constexpr int kPageWarps = kPageThreads / 32;
constexpr int kPageCluster = 8;      // the largest portable cluster
constexpr int kRowWords = 2048;      // bits for 65,536 rows

// Inclusive sum over the block's threads (`sums`: 32 values of shared memory); `total` gets the sum of all.
template <typename I> __device__ __forceinline__ I block_scan(I v, I *sums, I &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const I u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();                 // the sums of the call before have been read
    if (lane == 31) sums[warp] = v;
    __syncthreads();
    if (warp == 0) {
        I s = sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const I u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        sums[lane] = s;
    }
    __syncthreads();
    total = sums[kPageWarps - 1];
    return v + (warp > 0 ? sums[warp - 1] : 0);
}

// Which rows the active lanes (no entry negative) name, and which twice (whole block; every block for itself).
__device__ __forceinline__ void mark_rows(const int32_t *rows, const int32_t *active, int n, int n_rows, unsigned *seen, unsigned *twice) {
    for (int i = threadIdx.x; i < (n_rows + 31) / 32; i += blockDim.x) seen[i] = twice[i] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
        const int r = rows[i];
        if (r >= 0 && r < n_rows && active[i] >= 0) {
            const unsigned bit = 1u << (r & 31);
            if (atomicOr(seen + (r >> 5), bit) & bit) atomicOr(twice + (r >> 5), bit);
        }
    }
    __syncthreads();
}
__device__ __forceinline__ bool marked(const unsigned *bits, int r) { return bits[r >> 5] >> (r & 31) & 1u; }

// Row of a lane; -1: inactive, or reported and skipped.
__device__ __forceinline__ int lane_row(int r, const AttnDims &d, const unsigned *twice, unsigned *err) {
    if (r < 0) return -1;
    if (r >= d.n_rows || marked(twice, r)) {
        set_error(err, GDN_DEVERR_SLOT);
        return -1;
    }
    return r;
}

__device__ __forceinline__ int pages_of(int len, const AttnDims &d) { return (int)(((unsigned)len + d.page - 1) >> d.page_shift); }

// A page's index if it is one; else -1, reported.
__device__ __forceinline__ int checked(int page, const AttnDims &d, unsigned *err) {
    if (page >= 0 && page < d.n_pages) return page;
    set_error(err, GDN_DEVERR_PAGE);
    return -1;
}

// What a lane of a resize does, from the tables as they are when the call starts.
struct Resize {
    int row, old, len, have, want, last;     // last: the page that is copied, -1: none
    __device__ __forceinline__ int need() const { return max(want - have, 0) + (last >= 0); }
};
__device__ __forceinline__ Resize resize_lane(const PageArgs &a, int i, const unsigned *twice) {
    Resize r{-1, 0, 0, 0, 0, -1};
    const int new_len = a.new_lens[i];
    if (new_len < 0) return r;
    r.row = lane_row(a.rows[i], a.d, twice, a.err);
    if (r.row < 0) return r;
    const int most = a.d.max_pages * a.d.page;
    r.old = a.lens[r.row];
    if (r.old < 0 || r.old > most) {
        set_error(a.err, GDN_DEVERR_PAGE);
        r.old = min(max(r.old, 0), most);
    }
    r.len = new_len;
    if (r.len > most) {
        set_error(a.err, GDN_DEVERR_PAGE);
        r.len = r.old;
    }
    r.have = pages_of(r.old, a.d);
    r.want = pages_of(r.len, a.d);
    if (r.len > r.old && (r.old & (a.d.page - 1)) != 0) {
        const int page = checked(a.table[(long long)r.row * a.d.max_pages + r.have - 1], a.d, a.err);
        if (page >= 0 && a.refs[page] > 1) r.last = page;
    }
    return r;
}

// What a lane does once it is granted, as its warp finds it: in shared memory for the first kPageThreads lanes, where every
// CTA has them from its own sums; beyond, the place and the copied page come from the workspace, the rest again from the
// tables.
struct Lanes {
    int row[kPageThreads], old[kPageThreads], len[kPageThreads], last[kPageThreads], first[kPageThreads];
};

// Workspace: per lane the place of its first page among the free ones and the page that it copies; the free pages in order.
__global__ void __cluster_dims__(kPageCluster, 1, 1) __launch_bounds__(kPageThreads) page_resize_kernel(const PageArgs a) {
    extern __shared__ unsigned char raw[];
    Lanes &lanes = *reinterpret_cast<Lanes *>(raw);
    unsigned *seen = reinterpret_cast<unsigned *>(raw + sizeof(Lanes)), *twice = seen + kRowWords;
    __shared__ int sums[32], counted;
    __shared__ long long lane_sums[32];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, rank = (int)cluster.block_rank();
    int32_t *first = a.ws, *copied = a.ws + a.n, *fresh = a.ws + 2 * (size_t)a.n;
    await_previous();
    let_next_start();
    mark_rows(a.rows, a.new_lens, a.n, a.d.n_rows, seen, twice);
    // every CTA sums all lanes' needs; the first one writes the places of the lanes that shared memory does not hold
    long long needed = 0;
    for (int i0 = 0; i0 < a.n; i0 += kPageThreads) {
        const int i = i0 + tid;
        Resize r{-1, 0, 0, 0, 0, -1};
        if (i < a.n) r = resize_lane(a, i, twice);
        long long total;
        const long long upto = block_scan((long long)r.need(), lane_sums, total);
        // places behind the last page are no places: such a lane is not granted
        const int at = (int)min(needed + upto - r.need(), (long long)a.d.n_pages);
        if (i0 == 0) {
            lanes.row[tid] = r.row;
            lanes.old[tid] = r.old;
            lanes.len[tid] = r.len;
            lanes.last[tid] = r.last;
            lanes.first[tid] = at;
        } else if (rank == 0 && i < a.n) {
            first[i] = at;
            copied[i] = r.last;
        }
        needed += total;
    }
    // the free pages of this CTA's part of the counts, then their places among all
    int n_free = 0;
    if (needed > 0) {
        const int part = (((a.d.n_pages + kPageCluster - 1) / kPageCluster) + 3) & ~3;
        const int lo = min(part * rank, a.d.n_pages), hi = min(lo + part, a.d.n_pages);
        int mine = 0, total;
        for (int p = lo + tid; p < hi; p += kPageThreads) mine += a.refs[p] == 0;
        block_scan(mine, sums, total);
        if (tid == 0) counted = total;
        cluster.sync();
        int before = 0;
        for (int k = 0; k < kPageCluster; ++k) {
            const int c = *cluster.map_shared_rank(&counted, k);
            before += k < rank ? c : 0;
            n_free += c;
        }
        for (int p0 = lo; p0 < hi && before < needed; p0 += kPageThreads) {
            const int p = p0 + tid;
            const bool free = p < hi && a.refs[p] == 0;
            const int place = before + block_scan(free ? 1 : 0, sums, total) - 1;
            if (free && place < needed) fresh[place] = p;
            before += total;
        }
    }
    __threadfence();
    cluster.sync();                   // the lists are there, and all have read the tables as they were
    // a warp a lane
    for (int i = rank * kPageWarps + (tid >> 5); i < a.n; i += kPageCluster * kPageWarps) {
        const int lane = tid & 31;
        Resize r{-1, 0, 0, 0, 0, -1};
        int at;
        if (i < kPageThreads) {
            r.row = lanes.row[i];
            r.old = lanes.old[i];
            r.len = lanes.len[i];
            r.last = lanes.last[i];
            at = lanes.first[i];
        } else {
            // the counts have changed by now: what is copied was decided above
            at = first[i];
            const int row = a.rows[i], len = a.new_lens[i], most = a.d.max_pages * a.d.page;
            if (len >= 0 && row >= 0 && row < a.d.n_rows && !marked(twice, row)) {
                r.row = row;
                r.old = min(max(a.lens[row], 0), most);
                r.len = len > most ? r.old : len;
                r.last = copied[i];
            }
            __syncwarp();
        }
        r.have = pages_of(r.old, a.d);
        r.want = pages_of(r.len, a.d);
        const bool granted = r.row >= 0 && (r.need() == 0 || (long long)at + r.need() <= n_free);
        int place = at, to = -1;
        int32_t *entry = a.table + (long long)r.row * a.d.max_pages;
        if (granted && r.last >= 0) {
            to = fresh[place++];
            if (lane == 0) {
                entry[r.have - 1] = to;
                a.refs[to] = 1;
                atomicSub(a.refs + r.last, 1);
            }
        }
        if (granted) {
            for (int c = r.have + lane; c < r.want; c += 32) {
                const int p = fresh[place + c - r.have];
                entry[c] = p;
                a.refs[p] = 1;
            }
            for (int c = r.want + lane; c < r.have; c += 32) {
                const int p = checked(entry[c], a.d, a.err);
                if (p >= 0) atomicSub(a.refs + p, 1);
                entry[c] = -1;
            }
        }
        if (lane == 0) {
            if (granted) a.lens[r.row] = r.len;
            a.granted[i] = r.row < 0 ? -1 : granted ? r.len : r.old;
            a.src[i] = to >= 0 ? r.last : -1;
            a.dst[i] = to;
        }
    }
    // (no CTA reads another's shared memory behind the last cluster.sync)
}

constexpr int kForkThreads = 256;
__global__ void __launch_bounds__(kForkThreads) page_fork_kernel(const PageArgs a) {
    __shared__ unsigned seen[kRowWords], twice[kRowWords];
    await_previous();
    let_next_start();
    mark_rows(a.rows, a.new_lens, a.n, a.d.n_rows, seen, twice);
    const int lane = threadIdx.x & 31;
    for (int i = blockIdx.x * (kForkThreads / 32) + (threadIdx.x >> 5); i < a.n; i += gridDim.x * (kForkThreads / 32)) {
        const int to = a.rows[i], from = a.new_lens[i];
        if (to < 0 || from < 0) continue;
        if (to >= a.d.n_rows || from >= a.d.n_rows || marked(twice, to) || marked(seen, from) || a.lens[to] != 0) {
            set_error(a.err, GDN_DEVERR_SLOT);
            continue;
        }
        const int len = a.lens[from];
        if (len < 0 || len > a.d.max_pages * a.d.page) {
            set_error(a.err, GDN_DEVERR_PAGE);
            continue;
        }
        const int32_t *src = a.table + (long long)from * a.d.max_pages;
        int32_t *dst = a.table + (long long)to * a.d.max_pages;
        for (int c = lane; c < pages_of(len, a.d); c += 32) {
            const int p = src[c];
            if (checked(p, a.d, a.err) >= 0) atomicAdd(a.refs + p, 1);
            dst[c] = p;
        }
        __syncwarp();
        if (lane == 0) a.lens[to] = len;
    }
}

// Workspace: [0] held pages, then for every page its place after the moves.
__global__ void __cluster_dims__(kPageCluster, 1, 1) __launch_bounds__(kPageThreads) page_compact_kernel(const PageArgs a) {
    __shared__ int sums[32], counted[2];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, rank = (int)cluster.block_rank();
    int32_t *goes = a.ws + 1;
    await_previous();
    let_next_start();
    const int part = (a.d.n_pages + kPageCluster - 1) / kPageCluster;
    const int lo = min(part * rank, a.d.n_pages), hi = min(lo + part, a.d.n_pages);
    int held = 0, total;
    for (int p = lo + tid; p < hi; p += kPageThreads) held += a.refs[p] > 0;
    block_scan(held, sums, total);
    if (tid == 0) counted[0] = total;
    cluster.sync();
    int kept = 0, held_before = 0;
    for (int k = 0; k < kPageCluster; ++k) {
        const int c = *cluster.map_shared_rank(&counted[0], k);
        held_before += k < rank ? c : 0;
        kept += c;
    }
    // holes below `kept` in front of page p: p less the held ones in front; the held ones from `kept` on: held in front
    // less those below `kept`, of which there are kept - holes.  Holes and movers are as many.
    int below = 0;
    for (int p = lo + tid; p < min(hi, kept); p += kPageThreads) below += a.refs[p] > 0;
    block_scan(below, sums, total);
    if (tid == 0) counted[1] = total;
    cluster.sync();
    int stay = 0;
    for (int k = 0; k < kPageCluster; ++k) stay += *cluster.map_shared_rank(&counted[1], k);
    const int moves = min(kept - stay, a.n);
    // lists, ranks from the scan of held pages; the counts are read before any is written (refs_out may be refs)
    int running = held_before;
    for (int p0 = lo; p0 < hi; p0 += kPageThreads) {
        const int p = p0 + tid;
        const bool is = p < hi && a.refs[p] > 0;
        const int front = running + block_scan(is ? 1 : 0, sums, total) - (is ? 1 : 0);     // held pages in front of p
        running += total;
        if (p < hi) {
            goes[p] = p;
            if (p < kept && !is && p - front < moves) a.dst[p - front] = p;
            if (p >= kept && is && front - stay < moves) a.src[front - stay] = p;
        }
    }
    for (int i = moves + rank * kPageThreads + tid; i < a.n; i += kPageCluster * kPageThreads) a.src[i] = a.dst[i] = -1;
    if (rank == 0 && tid == 0) a.ws[0] = kept;
    if (a.refs_out != a.refs)
        for (int p = lo + tid; p < hi; p += kPageThreads) a.refs_out[p] = a.refs[p];
    __threadfence();
    cluster.sync();
    for (int i = rank * kPageThreads + tid; i < moves; i += kPageCluster * kPageThreads) {
        const int from = a.src[i], to = a.dst[i];
        goes[from] = to;
        a.refs_out[to] = a.refs[from];
        a.refs_out[from] = 0;
    }
    cluster.sync();
}

__global__ void __launch_bounds__(256) page_table_kernel(const PageArgs a) {
    let_next_start();
    await_previous();
    const long long all = (long long)a.d.n_rows * a.d.max_pages;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < all; i += (long long)gridDim.x * 256) {
        const int row = (int)(i / a.d.max_pages), c = (int)(i - (long long)row * a.d.max_pages);
        int p = a.table[i];
        const int len = min(max(a.lens[row], 0), a.d.max_pages * a.d.page);
        if (c < pages_of(len, a.d) && checked(p, a.d, a.err) >= 0) p = a.ws[1 + p];
        a.table_out[i] = p;
    }
}

// A block takes pieces of 16 KB; a piece is one of a page's, K's before V's.
constexpr int kCopyThreads = 256;
constexpr int kCopyPiece = 16384;
__global__ void __launch_bounds__(kCopyThreads) page_copy_kernel(const uint4 *src_k, const uint4 *src_v, int n_src, uint4 *dst_k, uint4 *dst_v,
                                                                 int n_dst, const int32_t *src_idx, const int32_t *dst_idx, int n,
                                                                 long long page_words, int pieces, unsigned *err) {
    const int per_lane = pieces * 2;
    let_next_start();
    await_previous();
    for (long long i = blockIdx.x; i < (long long)n * per_lane; i += gridDim.x) {
        const int lane = (int)(i / per_lane), k = (int)(i - (long long)lane * per_lane);
        const bool v = k >= pieces;
        const uint4 *from = v ? src_v : src_k;
        uint4 *to = v ? dst_v : dst_k;
        const int t = dst_idx[lane], s = src_idx[lane];
        if (t < 0 || !to) continue;
        if (t >= n_dst || (s >= n_src && from)) {
            set_error(err, GDN_DEVERR_PAGE);
            continue;
        }
        const long long w0 = (long long)(v ? k - pieces : k) * (kCopyPiece / 16), w1 = min(w0 + kCopyPiece / 16, page_words);
        to += t * page_words;
        if (s < 0 || !from) {
            for (long long w = w0 + threadIdx.x; w < w1; w += kCopyThreads) to[w] = make_uint4(0u, 0u, 0u, 0u);
        } else {
            from += s * page_words;
            for (long long w = w0 + threadIdx.x; w < w1; w += kCopyThreads) to[w] = from[w];
        }
    }
}

}  // namespace

size_t page_ws_ints(const AttnDims &d, long long lanes) { return 2 * (size_t)lanes + (size_t)d.n_pages + 4; }

cudaError_t launch_page_resize(const PageArgs &a, cudaStream_t s) {
    constexpr int smem = sizeof(Lanes) + 2 * kRowWords * 4;
    static_assert(smem <= 48 * 1024, "without opting in");
    return launch_early(page_resize_kernel, dim3(kPageCluster), kPageThreads, smem, s, a);
}

cudaError_t launch_page_fork(const PageArgs &a, cudaStream_t s) {
    const int blocks = (a.n + kForkThreads / 32 - 1) / (kForkThreads / 32), most = sm_count() * 4;
    return launch_early(page_fork_kernel, dim3(blocks < most ? blocks : most), kForkThreads, 0, s, a);
}

cudaError_t launch_page_compact(const PageArgs &a, cudaStream_t s) {
    const cudaError_t e = launch_early(page_compact_kernel, dim3(kPageCluster), kPageThreads, 0, s, a);
    if (e != cudaSuccess) return e;
    const long long all = (long long)a.d.n_rows * a.d.max_pages, blocks = (all + 255) / 256, most = (long long)sm_count() * 8;
    return launch_early(page_table_kernel, dim3((unsigned)(blocks < most ? blocks : most)), 256, 0, s, a);
}

cudaError_t launch_page_copy(const void *src_k, const void *src_v, int n_src, void *dst_k, void *dst_v, int n_dst,
                             const int32_t *src_idx, const int32_t *dst_idx, int n, long long page_bytes, unsigned *err,
                             cudaStream_t s) {
    const int pieces = (int)((page_bytes + kCopyPiece - 1) / kCopyPiece);
    const long long all = (long long)n * pieces * 2, most = (long long)sm_count() * 8;
    return launch_early(page_copy_kernel, dim3((unsigned)(all < most ? all : most)), kCopyThreads, 0, s, (const uint4 *)src_k, (const uint4 *)src_v,
                        n_src, (uint4 *)dst_k, (uint4 *)dst_v, n_dst, src_idx, dst_idx, n, page_bytes / 16, pieces, err);
}

}  // namespace gdn
