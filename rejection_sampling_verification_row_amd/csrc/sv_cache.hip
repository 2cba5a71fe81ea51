// Pages of a key-value cache around a verify step (gfx950).
//
// The state is the caller's: refs[page] counts a page's holders, and a page is free exactly when
// that is 0; a sequence holds tables[seq][0 .. blocks) and lengths[seq] tokens.  There is no free
// list whose order would depend on the history: a call that takes pages takes the lowest free
// ids, in list order, so its result is a function of the state alone.
//
// A call that takes pages is a plan and an apply.  The free pages are listed stretch by stretch of
// the pool, a workgroup each; one workgroup checks the list and prefix-sums what its entries ask
// for; then the whole chip writes the tables and copies pages.  The plan leaves for each entry one
// record of all that its apply needs, since an apply workgroup may find the state changed by
// another, and since a record is one trip to memory.
//
// The calls read and write little but for the copies, so they are bound by launches and by trips to
// memory in a row: a reserve and a commit of 512 sequences in a pool of 65536 pages take 4.6 us to
// list the free pages, 6.8 to plan, 3.7 to apply and 3.4 to commit.  Copies run at the rate of a
// large copy: a compaction that moves 696 pages of 8 x 32 KiB, 365 MB read and written by the
// counters, takes 69 us (5.3 TB/s); 2000 such pages copied, 1.05 GB, 203 us (5.2 TB/s); a fork of 480
// children, whose few sources stay in the caches, writes 67 MB in 13 us.
#include <algorithm>

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

// Bit k: page p + k is below end and free.
__device__ int free_bits(const CacheView &c, int p, int end)
{
    int bits = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (p + k < end && c.refs[p + k] == 0)
            bits |= 1 << k;
    return bits;
}

// The free pages of a stretch, ascending, into its part of free_ids.
__device__ void list_free(const CacheView &c, int stretch, int *lds)
{
    const int p = stretch * CACHE_STRETCH + (int)threadIdx.x * 4;
    static_assert(CACHE_STRETCH == CWG * 4, "four pages to a thread");
    const int bits = free_bits(c, p, c.num_pages);
    int all;
    int at = stretch * CACHE_STRETCH + block_incl_scan(__popc(bits), lds, &all) - __popc(bits);
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (bits >> k & 1)
            c.free_ids[at++] = p + k;
    if (threadIdx.x == 0)
        c.free_count[stretch] = all;
}

// Pools of more than one stretch list their free pages in a launch before the plan.
__global__ __launch_bounds__(CWG) void k_list_free(CacheView c)
{
    __shared__ int lds[CWAVES];
    list_free(c, blockIdx.x, lds);
}

// free_count becomes the free pages before each stretch, in LDS too as far as it holds them;
// returns how many there are.
constexpr int LDS_STRETCHES = 1024;

__device__ int scan_free(const CacheView &c, int stretches, int *before, int *lds)
{
    int sum = 0;
    for (int s0 = 0; s0 < stretches; s0 += CWG) {
        const int s = s0 + threadIdx.x, n = s < stretches ? c.free_count[s] : 0;
        int all;
        const int inc = block_incl_scan(n, lds, &all);
        if (s < stretches) {
            c.free_count[s] = sum + inc - n;
            if (s < LDS_STRETCHES)
                before[s] = sum + inc - n;
        }
        sum += all;
    }
    __syncthreads();
    return sum;
}

// The i-th free page: the last stretch with no more than i before it.
__device__ int free_page(const CacheView &c, int stretches, const int *before, int i)
{
    const bool small = stretches <= LDS_STRETCHES;
    int lo = 0, hi = stretches - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((small ? before[mid] : c.free_count[mid]) <= i)
            lo = mid;
        else
            hi = mid - 1;
    }
    const int at = i - (small ? before[lo] : c.free_count[lo]);
    return c.free_ids[lo * CACHE_STRETCH + at];
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
__device__ inline bool sound(const CacheView &c, int b, int l)
{
    return b >= 0 && b <= c.max_blocks && l >= 0 && l <= b * c.page_tokens;
}

// Gives the entries their places among the free pages, and lists the pages taken in c.map.
// ask(i, e) is what entry i asks for and fills in its record (-1: it is refused); an entry is
// granted when all that is asked up to it exists.  placed(e) then sees its record, seq -1 where
// nothing is granted.  Whole waves call both, past the list's end too.
template <typename Ask, typename Placed>
__device__ void grant(const CacheView &c, int n, int *status, int *lds, Ask ask, Placed placed)
{
    __shared__ int before[LDS_STRETCHES];
    const int stretches = (c.num_pages + CACHE_STRETCH - 1) / CACHE_STRETCH;
    if (stretches == 1) {
        list_free(c, 0, lds);
        __syncthreads();
    }
    const int found = scan_free(c, stretches, before, lds);
    // unsigned: sum stays at found + 1, 2^30 at most, and a tile asks for at most 1024 * 2^20
    uint32_t sum = 0;
    for (int i0 = 0; i0 < n; i0 += CWG) {
        const int i = i0 + threadIdx.x;
        CacheEntry e = {-1, -1, 0, 0, 0, 0, -1, -1};
        const int a = ask(i, e);
        int all;
        const int inc = block_incl_scan(max(a, 0), lds, &all);
        if (i < n) {
            const bool ok = a >= 0 && sum + (uint32_t)inc <= (uint32_t)found;
            e.first = (int)(sum + (uint32_t)(inc - a));
            if (!ok)
                e.seq = -1;
            else if (e.src >= 0)
                e.dst = free_page(c, stretches, before, e.first++);
            c.entries[i] = e;
            if (status)
                status[i] = ok ? 0 : -1;
        }
        placed(e);
        sum = min(sum + (uint32_t)all, (uint32_t)found + 1);
    }
    for (int i = threadIdx.x; i < (int)min(sum, (uint32_t)found); i += CWG)
        c.map[i] = free_page(c, stretches, before, i);
}

// How many of the blocks from .. to of a lane's sequence name a page that others hold too; with
// first >= 0 they are listed in c.src from there on.  A wave walks its lanes' blocks together, one
// lane's after another: few have any, since a commit leaves no page past the length.
__device__ int shared_blocks(const CacheView &c, int seq, int from, int to, int first)
{
    const int lane = threadIdx.x & 63;
    int mine = 0;
    for (uint64_t who = __ballot(from < to); who; who &= who - 1) {
        const int l = __builtin_ctzll(who), s = __shfl(seq, l), end = __shfl(to, l), at = __shfl(first, l);
        const int *row = c.tables + (size_t)s * c.max_blocks;
        int n = 0;
        for (int j0 = __shfl(from, l); j0 < end; j0 += 64) {
            const int j = j0 + lane, pg = j < end ? row[j] : -1;
            const bool shared = in_range(pg, c.num_pages) && c.refs[pg] > 1;
            const uint64_t all = __ballot(shared);
            if (shared && at >= 0)
                c.src[at + n + __popcll(all & ((1ull << lane) - 1))] = j;
            n += __popcll(all);
        }
        if (lane == l)
            mine = n;
    }
    return mine;
}

__global__ __launch_bounds__(CWG) void k_reserve_plan(CacheView c, int n, const int *seqs,
                                                      const int *counts, int *status)
{
    __shared__ int lds[CWAVES];
    claim(c, n, seqs);
    int past = 0, end = 0;         // the blocks held past the length that it will write into
    grant(
        c, n, status, lds,
        [&](int i, CacheEntry &e) {
            past = end = 0;
            int a = i < n ? -1 : 0;
            const int s = i < n ? (seqs ? seqs[i] : i) : -1, cnt = i < n ? counts[i] : 0;
            if (in_range(s, c.num_seqs) && load_agent(&c.owner[s]) == i) {
                const int len = c.lengths[s], had = c.blocks[s];
                if (sound(c, had, len) && cnt >= 0 && cnt <= c.max_blocks * c.page_tokens - len) {
                    e.seq = s;
                    e.had = e.want = had;
                    e.len = len;
                    a = 0;
                    if (cnt > 0) {
                        const int need = ceil_div(len + cnt, c.page_tokens);
                        e.want = max(had, need);
                        past = ceil_div(len, c.page_tokens);
                        end = min(had, need);
                        if (len % c.page_tokens != 0) {
                            // partly filled: a copy, where another holds it too
                            const int pg = c.tables[(size_t)s * c.max_blocks + len / c.page_tokens];
                            if (in_range(pg, c.num_pages) && c.refs[pg] > 1)
                                e.src = pg;
                        }
                        a = e.want - had + (e.src >= 0);
                    }
                }
            }
            e.from = shared_blocks(c, s, past, end, -1);
            return a + e.from;
        },
        [&](const CacheEntry &e) {
            if (e.seq < 0 || e.from == 0)
                end = past;
            shared_blocks(c, e.seq, past, end, e.first);
        });
    unclaim(c, n, seqs);
}

// Copies the planned pages in every pool: 16 KiB of a page to a workgroup, which stands at (part of
// the page, pool, entries) and strides along each; pages(i, from, to) gives entry i's pages.  Few
// entries copy anything, so a wave reads 64 of them at once, one a lane, and walks those that do.
constexpr int COPY_WG = 256;
constexpr int COPY_STEP = COPY_WG * 16;       // bytes that a workgroup loads at once
constexpr int COPY_ITEM = 4 * COPY_STEP;

__device__ inline uint4 load16(const char *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ inline void store16(char *p, const uint4 &v) { *reinterpret_cast<uint4 *>(p) = v; }

__device__ inline void copy_page(const CacheView &c, int from, int to)
{
    for (int pool = blockIdx.y; pool < c.num_pools; pool += gridDim.y) {
        const char *a = c.pools[pool] + (int64_t)from * c.page_bytes;
        char *b = c.pools[pool] + (int64_t)to * c.page_bytes;
        for (int64_t o = (int64_t)blockIdx.x * COPY_ITEM + threadIdx.x * 16; o < c.page_bytes;
             o += (int64_t)gridDim.x * COPY_ITEM) {
            // four variables: an array of them would live in LDS
            const bool h1 = o + COPY_STEP < c.page_bytes, h2 = o + 2 * COPY_STEP < c.page_bytes,
                       h3 = o + 3 * COPY_STEP < c.page_bytes;
            const uint4 none = make_uint4(0, 0, 0, 0);
            const uint4 v0 = load16(a + o), v1 = h1 ? load16(a + o + COPY_STEP) : none,
                        v2 = h2 ? load16(a + o + 2 * COPY_STEP) : none,
                        v3 = h3 ? load16(a + o + 3 * COPY_STEP) : none;
            store16(b + o, v0);
            if (h1)
                store16(b + o + COPY_STEP, v1);
            if (h2)
                store16(b + o + 2 * COPY_STEP, v2);
            if (h3)
                store16(b + o + 3 * COPY_STEP, v3);
        }
    }
}

template <typename P> __device__ void copy_pages(const CacheView &c, int n, P pages)
{
    const int lane = threadIdx.x & 63;
    const int64_t step = 64 * (int64_t)gridDim.z;
    for (int64_t i0 = blockIdx.z; i0 < n; i0 += step) {
        const int64_t i = i0 + (int64_t)lane * gridDim.z;
        int from = -1, to = -1;
        if (i < n)
            pages((int)i, from, to);
        uint64_t copies = __ballot(in_range(from, c.num_pages) && in_range(to, c.num_pages));
        while (copies) {
            const int j = __builtin_ctzll(copies);
            copies &= copies - 1;
            copy_page(c, __shfl(from, j), __shfl(to, j));
        }
    }
}

__device__ void copy_entries(const CacheView &c, int n)
{
    copy_pages(c, n, [&](int i, int &from, int &to) {
        from = c.entries[i].src;
        to = c.entries[i].dst;
    });
}

// Workgroups of a copy's launch, and this one among them.
__device__ inline int copy_groups() { return gridDim.x * gridDim.y * gridDim.z; }
__device__ inline int copy_group()
{
    return (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
}

__device__ inline void release(const CacheView &c, int pg)
{
    if (in_range(pg, c.num_pages) && atomicSub(&c.refs[pg], 1) <= 0)
        atomicAdd(&c.refs[pg], 1);
}

// An entry's pages, one lane each: those in place of shared ones, then had .. want; and its copied
// page.
__device__ inline void take_pages(const CacheView &c, const CacheEntry &e, int *row)
{
    const int lane = threadIdx.x & 63;
    for (int i = lane; i < e.from + e.want - e.had; i += 64) {
        const int pg = c.map[e.first + i];
        const int j = i < e.from ? c.src[e.first + i] : e.had + i - e.from;
        if (i < e.from)
            release(c, row[j]);
        row[j] = pg;
        c.refs[pg] = 1;
    }
    if (lane == 0 && e.dst >= 0) {
        row[e.len / c.page_tokens] = e.dst;
        c.refs[e.dst] = 1;
        release(c, e.src);
    }
}

__global__ __launch_bounds__(COPY_WG) void k_reserve_apply(CacheView c, int n)
{
    const int lane = threadIdx.x & 63, waves = copy_groups() * (COPY_WG / 64);
    for (int i = copy_group() * (COPY_WG / 64) + (threadIdx.x >> 6); i < n; i += waves) {
        const CacheEntry e = c.entries[i];
        if (e.seq < 0)
            continue;
        int *row = c.tables + (size_t)e.seq * c.max_blocks;
        take_pages(c, e, row);
        if (lane == 0 && e.want > e.had)
            c.blocks[e.seq] = e.want;
    }
    copy_entries(c, n);
}

__global__ __launch_bounds__(CWG) void k_commit(CacheView c, int n, const int *seqs,
                                                const int *accepted, int *status)
{
    claim(c, n, seqs);
    for (int i = threadIdx.x; i < n; i += CWG) {
        const int s = seqs ? seqs[i] : i;
        bool ok = in_range(s, c.num_seqs) && load_agent(&c.owner[s]) == i;
        if (ok) {
            const int had = c.blocks[s], len = c.lengths[s], add = accepted[i];
            ok = sound(c, had, len) && add >= -1 && add < had * c.page_tokens - len;
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
    auto ask = [&](int i, CacheEntry &e) {
        if (i >= n)
            return 0;
        const int a = parents[i], b = children[i];
        if (!in_range(a, c.num_seqs) || !in_range(b, c.num_seqs) || a == b ||
            load_agent(&c.owner[b]) != i || c.blocks[b] != 0 || c.lengths[b] != 0)
            return -1;
        const int len = c.lengths[a];
        if (!sound(c, c.blocks[a], len))
            return -1;
        e.seq = b;
        e.from = a;
        e.len = len;
        e.had = e.want = ceil_div(len, c.page_tokens);
        if (len % c.page_tokens == 0)
            return 0;
        // a partly filled page is replaced whatever the table names, out of range without contents
        const int pg = c.tables[(size_t)a * c.max_blocks + e.had - 1];
        e.src = pg >= 0 ? pg : c.num_pages;
        return 1;
    };
    grant(c, n, status, lds, ask, [](const CacheEntry &) {});
    unclaim(c, n, children);
}

__global__ __launch_bounds__(COPY_WG) void k_fork_apply(CacheView c, int n)
{
    const int lane = threadIdx.x & 63, waves = copy_groups() * (COPY_WG / 64);
    for (int i = copy_group() * (COPY_WG / 64) + (threadIdx.x >> 6); i < n; i += waves) {
        const CacheEntry e = c.entries[i];
        if (e.seq < 0)
            continue;
        const int *from = c.tables + (size_t)e.from * c.max_blocks;
        int *row = c.tables + (size_t)e.seq * c.max_blocks;
        for (int j = lane; j < e.want; j += 64) {
            if (e.dst >= 0 && j == e.want - 1) {
                row[j] = e.dst;
                c.refs[e.dst] = 1;
            } else {
                const int pg = from[j];
                row[j] = pg;
                if (in_range(pg, c.num_pages))
                    atomicAdd(&c.refs[pg], 1);
            }
        }
        if (lane == 0) {
            c.blocks[e.seq] = e.want;
            c.lengths[e.seq] = e.len;
        }
    }
    copy_entries(c, n);
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

// Compaction: of U pages in use, the i-th at or past U moves to the i-th free page (of which h lie
// below U, as many as there are pages to move), so that the pages in use become 0 .. U - 1 with
// the fewest moves.  Where a page goes follows from the free pages before it alone, so every
// stretch is mapped by a workgroup of its own.
__device__ void map_stretch(const CacheView &c, int stretch, int stretches, const int *before, int base,
                            int used, int holes, int *page_map, int *lds)
{
    const int p = stretch * CACHE_STRETCH + (int)threadIdx.x * 4, bits = free_bits(c, p, c.num_pages);
    int all;
    int free_before = base + block_incl_scan(__popc(bits), lds, &all) - __popc(bits);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if (p + k >= c.num_pages)
            break;
        int to = -1;
        if (bits >> k & 1) {
            ++free_before;
        } else if (p + k < used) {
            to = p + k;
        } else {
            const int i = p + k - free_before - (used - holes);
            to = free_page(c, stretches, before, i);
            c.src[i] = p + k;
            c.dst[i] = to;
        }
        c.map[p + k] = to;
        if (page_map)
            page_map[p + k] = to;
    }
}

// Counts, and for a pool of one stretch the map as well.
__global__ __launch_bounds__(CWG) void k_compact_plan(CacheView c, int *page_map, int *num_used)
{
    __shared__ int lds[CWAVES];
    __shared__ int before[LDS_STRETCHES];
    const int stretches = (c.num_pages + CACHE_STRETCH - 1) / CACHE_STRETCH;
    if (stretches == 1) {
        list_free(c, 0, lds);
        __syncthreads();
    }
    const int used = c.num_pages - scan_free(c, stretches, before, lds);
    const int at = min(used / CACHE_STRETCH, stretches - 1);
    const int base = at < LDS_STRETCHES ? before[at] : c.free_count[at];
    int holes;
    block_incl_scan(__popc(free_bits(c, at * CACHE_STRETCH + (int)threadIdx.x * 4, used)), lds, &holes);
    holes += base;
    if (threadIdx.x == 0) {
        c.count[0] = holes;
        c.count[1] = used;
        if (num_used)
            *num_used = used;
    }
    if (stretches == 1)
        map_stretch(c, 0, 1, before, 0, used, holes, page_map, lds);
}

__global__ __launch_bounds__(CWG) void k_compact_map(CacheView c, int *page_map)
{
    __shared__ int lds[CWAVES];
    __shared__ int before[LDS_STRETCHES];
    const int stretches = gridDim.x;
    for (int s = threadIdx.x; s < min(stretches, LDS_STRETCHES); s += CWG)
        before[s] = c.free_count[s];
    map_stretch(c, blockIdx.x, stretches, before, c.free_count[blockIdx.x], c.count[1], c.count[0], page_map,
                lds);
}

__global__ __launch_bounds__(COPY_WG) void k_compact_apply(CacheView c)
{
    const int n = *c.count;
    const int64_t threads = (int64_t)copy_groups() * COPY_WG;
    const int64_t t = (int64_t)copy_group() * COPY_WG + threadIdx.x;
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
    copy_pages(c, n, [&](int i, int &from, int &to) {
        from = c.src[i];
        to = c.dst[i];
    });
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
    copy_pages(c, n, [&](int i, int &from, int &to) {
        from = c.src[i];
        to = c.dst[i];
    });
}

__global__ void k_cache_init(CacheView c)
{
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i < max(c.num_seqs, c.num_pages))
        c.owner[i] = CACHE_NO_OWNER;
}

hipError_t list_stretches(hipStream_t st, const CacheView &c)
{
    const int n = (c.num_pages + CACHE_STRETCH - 1) / CACHE_STRETCH;
    if (n > 1)
        k_list_free<<<n, CWG, 0, st>>>(c);
    return hipGetLastError();
}

// The launch of an apply over n entries: a workgroup for every part of a page in every pool, and
// entries until there are about 8 workgroups per compute unit.
dim3 apply_grid(const CacheView &c, int cus, int64_t n)
{
    const int64_t most = 8 * (int64_t)cus;
    const int64_t parts = std::max<int64_t>((c.page_bytes + COPY_ITEM - 1) / COPY_ITEM, 1);
    const int64_t x = std::min(parts, most);
    const int64_t y = std::min<int64_t>(std::max(c.num_pools, 1), most / x);
    const int64_t z = std::min<int64_t>(std::max<int64_t>(n, 1), most / x / y);
    return dim3((unsigned)x, (unsigned)y, (unsigned)z);
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
    hipError_t e = list_stretches(st, c);
    if (e != hipSuccess)
        return e;
    k_reserve_plan<<<1, CWG, 0, st>>>(c, n, seqs, counts, status);
    e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    k_reserve_apply<<<apply_grid(c, cus, n), COPY_WG, 0, st>>>(c, n);
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
    hipError_t e = list_stretches(st, c);
    if (e != hipSuccess)
        return e;
    k_fork_plan<<<1, CWG, 0, st>>>(c, n, parents, children, status);
    e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    k_fork_apply<<<apply_grid(c, cus, n), COPY_WG, 0, st>>>(c, n);
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
    const int stretches = (c.num_pages + CACHE_STRETCH - 1) / CACHE_STRETCH;
    hipError_t e = list_stretches(st, c);
    if (e != hipSuccess)
        return e;
    k_compact_plan<<<1, CWG, 0, st>>>(c, page_map, num_used);
    e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    if (stretches > 1) {
        k_compact_map<<<stretches, CWG, 0, st>>>(c, page_map);
        e = hipGetLastError();
        if (e != hipSuccess)
            return e;
    }
    k_compact_apply<<<apply_grid(c, cus, c.num_pages), COPY_WG, 0, st>>>(c);
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
