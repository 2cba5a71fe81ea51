// Pages of a key-value cache around a verify step (gfx950).
//
// The state is the caller's: refs[page] counts a page's holders, and a page is free exactly when
// that is 0; a sequence holds tables[seq][0 .. blocks) and lengths[seq] tokens.  There is no free
// list whose order would depend on the history: a call that takes pages takes the lowest free
// ids, in list order, so its result is a function of the state alone.
//
// A call that takes pages is a plan and an apply: one workgroup checks the list, prefix-sums what
// each entry asks for and finds the free ids; then the whole chip writes the tables and copies
// pages.  The plan keeps in scratch whatever an apply workgroup could find changed by another.
#include "sv_device.h"
#include "sv_internal.h"

namespace sv {

namespace {

constexpr int CWG = 1024;
constexpr int CWAVES = CWG / 64;

__device__ inline bool in_range(int i, int n) { return (unsigned)i < (unsigned)n; }
__device__ inline int ceil_div(int a, int b) { return a / b + (a % b != 0); }

__device__ inline int load_agent(const int *p)
{
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ inline int wave_incl_scan_int(int v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(v, o);
        if (lane >= o)
            v += u;
    }
    return v;
}

// Inclusive scan over the workgroup in thread order; *total is the sum.
__device__ inline int block_incl_scan(int v, int *lds, int *total)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int inc = wave_incl_scan_int(v);
    __syncthreads();
    if (lane == 63)
        lds[w] = inc;
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < CWAVES; ++i) {
        before += i < w ? lds[i] : 0;
        all += lds[i];
    }
    *total = all;
    return before + inc;
}

// The first `want` free pages, ascending, into ids (fewer if there are fewer); returns how many.
__device__ int find_free(const CacheView &c, int want, int *ids, int *lds)
{
    int found = 0;
    for (int p0 = 0; p0 < c.num_pages && found < want; p0 += CWG * 4) {
        const int p = p0 + (int)threadIdx.x * 4;
        int bits = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (p + k < c.num_pages && c.refs[p + k] == 0)
                bits |= 1 << k;
        int all;
        int at = found + block_incl_scan(__popc(bits), lds, &all) - __popc(bits);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (bits >> k & 1) {
                if (at < want)
                    ids[at] = p + k;
                ++at;
            }
        found += all;
    }
    return min(found, want);
}

// The list entries that name a sequence first own it; later ones are refused.
__device__ void claim(const CacheView &c, int n, const int *seqs)
{
    for (int i = threadIdx.x; i < n; i += CWG) {
        const int s = seqs ? seqs[i] : i;
        if (in_range(s, c.num_seqs))
            atomicMin(&c.owner[s], i);
    }
    __syncthreads();
}

__device__ void unclaim(const CacheView &c, int n, const int *seqs)
{
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += CWG) {
        const int s = seqs ? seqs[i] : i;
        if (in_range(s, c.num_seqs))
            c.owner[s] = CACHE_NO_OWNER;
    }
}

// an entry's sequence has a state that an operation may build on
__device__ inline bool sound(const CacheView &c, int s)
{
    const int b = c.blocks[s], l = c.lengths[s];
    return b >= 0 && b <= c.max_blocks && l >= 0 && l <= b * c.page_tokens;
}

// Gives the entries their places among the free pages.  ask(i) is what entry i asks for (-1: it
// is refused); an entry is granted when all that is asked up to it exists.
template <typename Ask>
__device__ void grant(const CacheView &c, int n, int *status, int *lds, Ask ask)
{
    int sum = 0;
    for (int i0 = 0; i0 < n; i0 += CWG) {
        const int i = i0 + threadIdx.x;
        const int a = i < n ? ask(i) : 0;
        int all;
        // no overflow: an entry asks for at most max_blocks + 1 pages, which is at most 2^20 + 1
        const int inc = block_incl_scan(max(a, 0), lds, &all);
        if (i < n)
            c.off[i] = a < 0 ? -1 : sum + inc - a;
        sum = min(sum + all, c.num_pages + 1);
    }
    __syncthreads();
    const int found = find_free(c, min(sum, c.num_pages), c.free_ids, lds);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += CWG) {
        const int o = c.off[i];
        const bool ok = o >= 0 && o + ask(i) <= found;
        c.off[i] = ok ? o : -1;
        if (status)
            status[i] = ok ? 0 : -1;
    }
}

// Reserve: entry i needs pages for lengths + counts tokens, and a page of its own where it will
// write into a partly filled page that another holds too.
__device__ inline bool needs_own(const CacheView &c, int s, int len)
{
    if (len % c.page_tokens == 0)
        return false;
    const int pg = c.tables[(size_t)s * c.max_blocks + len / c.page_tokens];
    return in_range(pg, c.num_pages) && c.refs[pg] > 1;
}

__global__ __launch_bounds__(CWG) void k_reserve_plan(CacheView c, int n, const int *seqs,
                                                      const int *counts, int *status)
{
    __shared__ int lds[CWAVES];
    claim(c, n, seqs);
    auto ask = [&](int i) {
        const int s = seqs ? seqs[i] : i;
        if (!in_range(s, c.num_seqs) || load_agent(&c.owner[s]) != i || !sound(c, s))
            return -1;
        const int len = c.lengths[s], cnt = counts[i];
        if (cnt < 0 || cnt > c.max_blocks * c.page_tokens - len)
            return -1;
        if (cnt == 0)
            return 0;
        return max(0, ceil_div(len + cnt, c.page_tokens) - c.blocks[s]) + (int)needs_own(c, s, len);
    };
    grant(c, n, status, lds, ask);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += CWG) {
        const int s = seqs ? seqs[i] : i;
        int from = -1, to = -1;
        if (c.off[i] >= 0 && counts[i] > 0 && needs_own(c, s, c.lengths[s])) {
            from = c.tables[(size_t)s * c.max_blocks + c.lengths[s] / c.page_tokens];
            to = c.free_ids[c.off[i]];
        }
        c.src[i] = from;
        c.dst[i] = to;
    }
    unclaim(c, n, seqs);
}

// Copies the planned pages in every pool.  A work item is 16 KiB of one page in one pool; the
// workgroups take items at a stride.
constexpr int COPY_WG = 256;
constexpr int COPY_VECS = 4;
constexpr int COPY_ITEM = COPY_WG * COPY_VECS * 16;

__device__ void copy_pages(const CacheView &c, int n, const int *src, const int *dst)
{
    const int per = (int)((c.page_bytes + COPY_ITEM - 1) / COPY_ITEM);
    const int64_t items = (int64_t)n * c.num_pools * per;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int part = (int)(it % per);
        const int64_t rest = it / per;
        const int pool = (int)(rest % c.num_pools), i = (int)(rest / c.num_pools);
        const int from = src[i], to = dst[i];
        if (!in_range(from, c.num_pages) || !in_range(to, c.num_pages))
            continue;
        const char *a = c.pools[pool] + (int64_t)from * c.page_bytes;
        char *b = c.pools[pool] + (int64_t)to * c.page_bytes;
        const int64_t o = (int64_t)part * COPY_ITEM + (int64_t)threadIdx.x * 16;
        uint4 v[COPY_VECS];
#pragma unroll
        for (int k = 0; k < COPY_VECS; ++k)
            if (o + k * COPY_WG * 16 < c.page_bytes)
                v[k] = *reinterpret_cast<const uint4 *>(a + o + k * COPY_WG * 16);
#pragma unroll
        for (int k = 0; k < COPY_VECS; ++k)
            if (o + k * COPY_WG * 16 < c.page_bytes)
                *reinterpret_cast<uint4 *>(b + o + k * COPY_WG * 16) = v[k];
    }
}

__global__ __launch_bounds__(COPY_WG) void k_reserve_apply(CacheView c, int n, const int *seqs,
                                                           const int *counts)
{
    const int lane = threadIdx.x & 63, waves = gridDim.x * (COPY_WG / 64);
    for (int i = blockIdx.x * (COPY_WG / 64) + (threadIdx.x >> 6); i < n; i += waves) {
        int o = c.off[i];
        if (o < 0 || counts[i] == 0)
            continue;
        const int s = seqs ? seqs[i] : i;
        const int len = c.lengths[s], had = c.blocks[s];
        const int want = ceil_div(len + counts[i], c.page_tokens);
        int *row = c.tables + (size_t)s * c.max_blocks;
        if (c.dst[i] >= 0) {
            if (lane == 0) {
                row[len / c.page_tokens] = c.dst[i];
                c.refs[c.dst[i]] = 1;
                atomicSub(&c.refs[c.src[i]], 1);
            }
            ++o;
        }
        for (int j = had + lane; j < want; j += 64) {
            const int pg = c.free_ids[o + j - had];
            row[j] = pg;
            c.refs[pg] = 1;
        }
        if (lane == 0 && want > had)
            c.blocks[s] = want;
    }
    copy_pages(c, n, c.src, c.dst);
}

__device__ inline void release(const CacheView &c, int pg)
{
    if (in_range(pg, c.num_pages) && atomicSub(&c.refs[pg], 1) <= 0)
        atomicAdd(&c.refs[pg], 1);
}

__global__ __launch_bounds__(CWG) void k_commit(CacheView c, int n, const int *seqs,
                                                const int *accepted, int *status)
{
    claim(c, n, seqs);
    for (int i = threadIdx.x; i < n; i += CWG) {
        const int s = seqs ? seqs[i] : i;
        bool ok = in_range(s, c.num_seqs) && load_agent(&c.owner[s]) == i && sound(c, s);
        if (ok) {
            const int had = c.blocks[s], len = c.lengths[s], add = accepted[i];
            ok = add >= -1 && add < had * c.page_tokens - len;
            if (ok) {
                const int left = ceil_div(len + add + 1, c.page_tokens);
                int *row = c.tables + (size_t)s * c.max_blocks;
                for (int j = left; j < had; ++j) {
                    release(c, row[j]);
                    row[j] = -1;
                }
                c.blocks[s] = left;
                c.lengths[s] = len + add + 1;
            }
        }
        if (status)
            status[i] = ok ? 0 : -1;
    }
    unclaim(c, n, seqs);
}

__global__ __launch_bounds__(CWG) void k_fork_plan(CacheView c, int n, const int *parents,
                                                   const int *children, int *status)
{
    __shared__ int lds[CWAVES];
    claim(c, n, children);
    auto ask = [&](int i) {
        const int a = parents[i], b = children[i];
        if (!in_range(a, c.num_seqs) || !in_range(b, c.num_seqs) || a == b ||
            load_agent(&c.owner[b]) != i || c.blocks[b] != 0 || c.lengths[b] != 0 || !sound(c, a))
            return -1;
        return (int)(c.lengths[a] % c.page_tokens != 0);
    };
    grant(c, n, status, lds, ask);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += CWG) {
        int from = -1, to = -1;
        if (c.off[i] >= 0) {
            const int a = parents[i], len = c.lengths[a];
            c.len[i] = len;
            if (len % c.page_tokens != 0) {
                from = c.tables[(size_t)a * c.max_blocks + len / c.page_tokens];
                to = c.free_ids[c.off[i]];
            }
        }
        c.src[i] = from;
        c.dst[i] = to;
    }
    unclaim(c, n, children);
}

__global__ __launch_bounds__(COPY_WG) void k_fork_apply(CacheView c, int n, const int *parents,
                                                        const int *children)
{
    const int lane = threadIdx.x & 63, waves = gridDim.x * (COPY_WG / 64);
    for (int i = blockIdx.x * (COPY_WG / 64) + (threadIdx.x >> 6); i < n; i += waves) {
        if (c.off[i] < 0)
            continue;
        const int len = c.len[i], nb = ceil_div(len, c.page_tokens), to = c.dst[i];
        const int *from = c.tables + (size_t)parents[i] * c.max_blocks;
        int *row = c.tables + (size_t)children[i] * c.max_blocks;
        for (int j = lane; j < nb; j += 64) {
            if (to >= 0 && j == nb - 1) {
                row[j] = to;
                c.refs[to] = 1;
            } else {
                const int pg = from[j];
                row[j] = pg;
                if (in_range(pg, c.num_pages))
                    atomicAdd(&c.refs[pg], 1);
            }
        }
        if (lane == 0) {
            c.blocks[children[i]] = nb;
            c.lengths[children[i]] = len;
        }
    }
    copy_pages(c, n, c.src, c.dst);
}

// One wave per entry.  The exchange lets only one of several entries that name a sequence see its
// pages.
__global__ __launch_bounds__(COPY_WG) void k_free(CacheView c, int n, const int *seqs,
                                                  const uint8_t *keep)
{
    const int i = blockIdx.x * (COPY_WG / 64) + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (i >= n || (keep && keep[i]))
        return;
    const int s = seqs ? seqs[i] : i;
    if (!in_range(s, c.num_seqs))
        return;
    int had = 0;
    if (lane == 0) {
        had = atomicExch(&c.blocks[s], 0);
        c.lengths[s] = 0;
    }
    had = min(__shfl(had, 0), c.max_blocks);
    int *row = c.tables + (size_t)s * c.max_blocks;
    for (int j = lane; j < had; j += 64) {
        release(c, row[j]);
        row[j] = -1;
    }
}

// Compaction: of U used pages, the i-th used page at or past U moves to the i-th free page below
// U, so that the used pages become 0 .. U - 1 with the fewest moves.
__global__ __launch_bounds__(CWG) void k_compact_plan(CacheView c, int *page_map, int *num_used)
{
    __shared__ int lds[CWAVES];
    int mine = 0, used = 0;
    for (int p = threadIdx.x; p < c.num_pages; p += CWG)
        mine += c.refs[p] > 0;
    block_incl_scan(mine, lds, &used);
    int holes = 0, movers = 0;
    for (int p0 = 0; p0 < c.num_pages; p0 += CWG) {
        const int p = p0 + threadIdx.x;
        const bool there = p < c.num_pages, full = there && c.refs[p] > 0;
        const bool hole = there && !full && p < used, mover = full && p >= used;
        int h, m;
        const int ih = holes + block_incl_scan(hole, lds, &h);
        const int im = movers + block_incl_scan(mover, lds, &m);
        if (hole)
            c.dst[ih - 1] = p;
        if (mover)
            c.src[im - 1] = p;
        if (there)
            c.map[p] = full ? p : -1;
        holes += h;
        movers += m;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < movers; i += CWG)
        c.map[c.src[i]] = c.dst[i];
    __syncthreads();
    if (page_map)
        for (int p = threadIdx.x; p < c.num_pages; p += CWG)
            page_map[p] = c.map[p];
    if (threadIdx.x == 0) {
        *c.count = movers;
        if (num_used)
            *num_used = used;
    }
}

__global__ __launch_bounds__(COPY_WG) void k_compact_apply(CacheView c)
{
    const int n = *c.count;
    const int64_t threads = (int64_t)gridDim.x * COPY_WG;
    const int64_t t = (int64_t)blockIdx.x * COPY_WG + threadIdx.x;
    for (int64_t i = t; i < n; i += threads) {
        c.refs[c.dst[i]] = c.refs[c.src[i]];
        c.refs[c.src[i]] = 0;
    }
    if (n > 0)
        for (int64_t e = t; e < (int64_t)c.num_seqs * c.max_blocks; e += threads) {
            const int pg = c.tables[e];
            if (in_range(pg, c.num_pages) && c.map[pg] != pg)
                c.tables[e] = c.map[pg];
        }
    copy_pages(c, n, c.src, c.dst);
}

// Copy: an entry is refused if a page is out of range, its destination is an earlier entry's, or
// its source is any entry's destination (so that no copy reads what another writes).
__global__ __launch_bounds__(CWG) void k_copy_plan(CacheView c, int n, const int *src,
                                                   const int *dst, int *status)
{
    for (int i = threadIdx.x; i < n; i += CWG)
        if (in_range(dst[i], c.num_pages))
            atomicMin(&c.owner[dst[i]], i);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += CWG) {
        const int a = src[i], b = dst[i];
        const bool ok = in_range(a, c.num_pages) && in_range(b, c.num_pages) &&
                        load_agent(&c.owner[b]) == i && load_agent(&c.owner[a]) == CACHE_NO_OWNER;
        c.src[i] = ok ? a : -1;
        c.dst[i] = ok ? b : -1;
        if (status)
            status[i] = ok ? 0 : -1;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += CWG)
        if (in_range(dst[i], c.num_pages))
            c.owner[dst[i]] = CACHE_NO_OWNER;
}

__global__ __launch_bounds__(COPY_WG) void k_copy_apply(CacheView c, int n)
{
    copy_pages(c, n, c.src, c.dst);
}

__global__ void k_cache_init(CacheView c)
{
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < max(c.num_seqs, c.num_pages))
        c.owner[i] = CACHE_NO_OWNER;
}

// workgroups of an apply: one per copy item up to 8 per compute unit, and at least one wave per
// four list entries
int apply_grid(const CacheView &c, int cus, int64_t n)
{
    const int64_t per = (c.page_bytes + COPY_ITEM - 1) / COPY_ITEM;
    const int64_t items = n * c.num_pools * per;
    const int64_t least = (n + COPY_WG / 64 - 1) / (COPY_WG / 64);
    const int64_t g = items > least ? items : least;
    return (int)(g < 8 * (int64_t)cus ? (g > 0 ? g : 1) : 8 * (int64_t)cus);
}

}  // namespace

hipError_t launch_cache_init(hipStream_t st, const CacheView &c)
{
    const int n = c.num_seqs > c.num_pages ? c.num_seqs : c.num_pages;
    k_cache_init<<<(n + 255) / 256, 256, 0, st>>>(c);
    return hipGetLastError();
}

hipError_t launch_cache_reserve(hipStream_t st, const CacheView &c, int cus, int n, const int *seqs,
                                const int *counts, int *status)
{
    k_reserve_plan<<<1, CWG, 0, st>>>(c, n, seqs, counts, status);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    k_reserve_apply<<<apply_grid(c, cus, n), COPY_WG, 0, st>>>(c, n, seqs, counts);
    return hipGetLastError();
}

hipError_t launch_cache_commit(hipStream_t st, const CacheView &c, int n, const int *seqs,
                               const int *accepted, int *status)
{
    k_commit<<<1, CWG, 0, st>>>(c, n, seqs, accepted, status);
    return hipGetLastError();
}

hipError_t launch_cache_fork(hipStream_t st, const CacheView &c, int cus, int n,
                             const int *parents, const int *children, int *status)
{
    k_fork_plan<<<1, CWG, 0, st>>>(c, n, parents, children, status);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    k_fork_apply<<<apply_grid(c, cus, n), COPY_WG, 0, st>>>(c, n, parents, children);
    return hipGetLastError();
}

hipError_t launch_cache_free(hipStream_t st, const CacheView &c, int n, const int *seqs,
                             const uint8_t *keep)
{
    k_free<<<(n + COPY_WG / 64 - 1) / (COPY_WG / 64), COPY_WG, 0, st>>>(c, n, seqs, keep);
    return hipGetLastError();
}

hipError_t launch_cache_compact(hipStream_t st, const CacheView &c, int cus, int *page_map,
                                int *num_used)
{
    k_compact_plan<<<1, CWG, 0, st>>>(c, page_map, num_used);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    k_compact_apply<<<8 * cus, COPY_WG, 0, st>>>(c);
    return hipGetLastError();
}

hipError_t launch_cache_copy(hipStream_t st, const CacheView &c, int cus, int n, const int *src,
                             const int *dst, int *status)
{
    k_copy_plan<<<1, CWG, 0, st>>>(c, n, src, dst, status);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    k_copy_apply<<<apply_grid(c, cus, n), COPY_WG, 0, st>>>(c, n);
    return hipGetLastError();
}

}  // namespace sv
