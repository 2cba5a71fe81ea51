// Greedy verify of a drafted tree, and the move of its accepted path in a cache (gfx950).
//
// The walk needs the argmax of one row a depth.  All rows at once is one launch that reads
// everything and a launch that walks; depth by depth is a launch for each depth, which reads one row
// of each sequence that is still walking.  In a launch of the latter every workgroup merges its
// sequence's partials of the depth before, finds the next node and reads its chunk of that row, so
// that no workgroup waits for another.  Trees whose rows are short take one launch: a workgroup has one.
#include <algorithm>
#include <limits.h>

#include "sv_internal.h"
#include "sv_memory.h"
#include "sv_tree.h"

namespace sv {

namespace {

__device__ inline bool in_range(int i, int n) { return (unsigned)i < (unsigned)n; }

// The lowest id of a row's maximum from its chunks' partials; whole waves.
__device__ inline int merge_partials(const float2 *part, int np)
{
    float v = -INFINITY;
    int id = INT_MAX;
    for (int i = threadIdx.x & 63; i < np; i += 64) {
        const float2 e = part[i];
        take_better(v, id, e.x, __float_as_int(e.y));
    }
    wave_argmax(v, id);
    return id;
}

// A tree's nodes, one to a lane; sound: its count, ids and parents are.
struct Nodes {
    int token, parent, count;
    bool sound;
};

__device__ inline Nodes load_nodes(const int *tokens, const int *parents, const int *counts, int b, int T, int V)
{
    const int lane = threadIdx.x & 63;
    Nodes n = {-1, -1, counts ? counts[b] : T, false};
    const bool good = n.count >= 1 && n.count <= T;
    bool bad = false;
    if (good && lane > 0 && lane < n.count) {
        n.token = tokens[(size_t)b * T + lane];
        n.parent = parents[(size_t)b * T + lane];
        bad = !in_range(n.token, V) || !in_range(n.parent, lane);
    }
    n.sound = good && __ballot(bad) == 0;
    return n;
}

// The lowest child of node `at` that holds id g, -1 if none.
__device__ inline int child_of(const Nodes &n, int at, int g)
{
    const uint64_t fits = __ballot(n.parent == at && n.token == g && (threadIdx.x & 63) > 0);
    return fits ? __builtin_ctzll(fits) : -1;
}

// All rows are reduced: one wave walks a sequence.
__global__ __launch_bounds__(64) void k_tree_walk(const int *tokens, const int *parents, const int *counts, int T,
                                                  int V, int depth, int np, const float2 *part, int *acc,
                                                  int *path, int *out)
{
    const int b = blockIdx.x, lane = threadIdx.x;
    const Nodes n = load_nodes(tokens, parents, counts, b, T, V);
    int at = 0, L = -1, my_node = -1, my_token = -1;
    while (n.sound && at >= 0) {
        const int g = merge_partials(part + ((size_t)b * T + at) * np, np);
        ++L;
        if (lane == L) {
            my_node = at;
            my_token = g;
        }
        at = L < depth ? child_of(n, at, g) : -1;
    }
    if (lane <= depth) {
        path[(size_t)b * (depth + 1) + lane] = my_node;
        out[(size_t)b * (depth + 1) + lane] = my_token;
    }
    if (lane == 0)
        acc[b] = L;
}

// 16 bytes of a row from id e on, at any address of the element's alignment.
template <int DT> __device__ inline u32x4 load_group(const char *row, int e)
{
    return load_once<u32x4_any>(row + (size_t)e * Elt<DT>::BYTES);
}
template <int DT> __device__ inline u32x4 low_group()
{
    const uint32_t low = DT == 1 ? 0xff80ff80u : 0xff800000u;
    return u32x4{low, low, low, low};
}
// The group that holds the row's last id.
template <int DT> __device__ inline u32x4 end_group(const char *row, int e, int V)
{
    u32x4 v = low_group<DT>();
#pragma unroll
    for (int k = 0; k < Elt<DT>::EPV; ++k)
        if (e + k < V) {
            const uint32_t x = __float_as_uint(Elt<DT>::one(row, e + k));
            if constexpr (DT == 0)
                v[k] = x;
            else
                v[k / 2] = k & 1 ? (v[k / 2] & 0xffffu) | x : (v[k / 2] & 0xffff0000u) | x >> 16;
        }
    return v;
}

// Chunk c of a row: each wave's maximum and the lowest id that has it.
template <int DT> __device__ __forceinline__ void chunk_best(const char *row, int V, int c, float2 *to)
{
    constexpr int E = Elt<DT>::EPV;
    const int t = threadIdx.x;
    const int base = c * WG * NV_ARGMAX * E;
    u32x4 raw[NV_ARGMAX];
    if (base + WG * NV_ARGMAX * E <= V) {
#pragma unroll
        for (int i = 0; i < NV_ARGMAX; ++i)
            raw[i] = load_group<DT>(row, base + (i * WG + t) * E);
    } else {
        // the row's end: what is past it reads as -inf
#pragma unroll
        for (int i = 0; i < NV_ARGMAX; ++i) {
            const int e = base + (i * WG + t) * E;
            raw[i] = e + E <= V ? load_group<DT>(row, e) : low_group<DT>();
            if (e < V && e + E > V)
                raw[i] = end_group<DT>(row, e, V);
        }
    }
    float bv = -INFINITY;
    int bi = base + t * E < V ? base + t * E : INT_MAX;
#pragma unroll
    for (int i = 0; i < NV_ARGMAX; ++i) {
        float x[E];
        Elt<DT>::unpack(make_uint4(raw[i][0], raw[i][1], raw[i][2], raw[i][3]), x);
#pragma unroll
        for (int k = 0; k < E; ++k)
            if (x[k] > bv) {
                bv = x[k];
                bi = base + (i * WG + t) * E + k;
            }
    }
    wave_argmax(bv, bi);
    if ((t & 63) == 0)
        to[t >> 6] = make_float2(bv, __int_as_float(bi));
}

// All rows, a workgroup to a chunk.
template <int DT>
__global__ __launch_bounds__(WG) void k_tree_rows(const char *__restrict__ tgt, int V, int nch, float2 *part)
{
    const size_t r = blockIdx.x / nch;
    chunk_best<DT>(tgt + r * (size_t)V * Elt<DT>::BYTES, V, (int)(blockIdx.x - r * nch),
                   part + (size_t)blockIdx.x * WAVES);
}

// A whole tree: each wave the argmaxes of every TREE_WAVES-th row, then the walk.  Bound by the call for a
// few short rows (one tree of 8 nodes, 1000 ids: 8.2 us, of which the host's 8), by what a compute unit reads else
// (256 trees of 64 nodes, 4000 ids, bfloat16: 23 us, 5.7 TB/s; all rows first: 53 us).
constexpr int TREE_LOADS = 4;
template <int DT>
__global__ __launch_bounds__(64 * TREE_WAVES) void k_tree_short(const char *__restrict__ tgt, const int *tokens,
                                                                const int *parents, const int *counts, int T, int V,
                                                                int depth, int *acc, int *path, int *out)
{
    constexpr int E = Elt<DT>::EPV;
    __shared__ int best[MAX_NODES];
    const int b = blockIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const Nodes n = load_nodes(tokens, parents, counts, b, T, V);
    for (int i = w; i < T && n.sound && i < n.count; i += blockDim.x >> 6) {
        const char *row = tgt + ((size_t)b * T + i) * (size_t)V * Elt<DT>::BYTES;
        float bv = -INFINITY;
        int bi = lane * E < V ? lane * E : INT_MAX;
        for (int base = 0; base < V; base += 64 * E * TREE_LOADS) {
            u32x4 raw[TREE_LOADS];
#pragma unroll
            for (int k = 0; k < TREE_LOADS; ++k) {
                const int e = base + (k * 64 + lane) * E;
                raw[k] = e + E <= V ? load_group<DT>(row, e) : low_group<DT>();
                if (e < V && e + E > V)
                    raw[k] = end_group<DT>(row, e, V);
            }
#pragma unroll
            for (int k = 0; k < TREE_LOADS; ++k) {
                float x[E];
                Elt<DT>::unpack(make_uint4(raw[k][0], raw[k][1], raw[k][2], raw[k][3]), x);
#pragma unroll
                for (int j = 0; j < E; ++j)
                    if (x[j] > bv) {
                        bv = x[j];
                        bi = base + (k * 64 + lane) * E + j;
                    }
            }
        }
        wave_argmax(bv, bi);
        if (lane == 0)
            best[i] = bi;
    }
    __syncthreads();
    if (w > 0)
        return;
    int at = n.sound ? 0 : -1, L = -1, my_node = -1, my_token = -1;
    while (at >= 0) {
        const int g = best[at];
        ++L;
        if (lane == L) {
            my_node = at;
            my_token = g;
        }
        at = L < depth ? child_of(n, at, g) : -1;
    }
    if (lane <= depth) {
        path[(size_t)b * (depth + 1) + lane] = my_node;
        out[(size_t)b * (depth + 1) + lane] = my_token;
    }
    if (lane == 0)
        acc[b] = L;
}

// One depth of every walk, `groups` workgroups to a sequence.  Workgroup (b, c): the node that the walk
// stands on after the `level` tokens before (from the row that the launch before reduced), and chunk c
// of its row.  The sequence's first workgroup writes what is known.  Partials alternate between two
// halves, since others of the sequence may still read those before.
//
// Bound by the launches, which wait for one another: 64 trees, depth 8, 128256 ids in bfloat16: 10
// launches, 49 us, of which 16 us go to at most 148 MB of rows.
template <int DT>
__global__ __launch_bounds__(WG) void k_tree_level(const char *__restrict__ tgt, const int *tokens,
                                                   const int *parents, const int *counts, int T, int V, int depth,
                                                   int level, int groups, int nch, const float2 *before,
                                                   float2 *part, int *acc, int *path, int *out)
{
    const int b = blockIdx.x / groups, c = blockIdx.x - b * groups, t = threadIdx.x;
    int *p = path + (size_t)b * (depth + 1), *o = out + (size_t)b * (depth + 1);
    const Nodes n = load_nodes(tokens, parents, counts, b, T, V);
    const bool first = c == 0 && t == 0;
    int at = n.sound ? 0 : -1;
    if (level > 0) {
        const int prev = p[level - 1];
        int g = -1;
        at = -1;
        if (prev >= 0) {
            g = merge_partials(before + (size_t)b * nch * WAVES, nch * WAVES);
            at = level <= depth ? child_of(n, prev, g) : -1;
        }
        if (first) {
            o[level - 1] = g;
            if (prev >= 0 && at < 0)
                acc[b] = level - 1;
        }
    } else if (first && at < 0) {
        acc[b] = -1;
    }
    if (first && level <= depth)
        p[level] = at;
    if (at < 0)
        return;
    const char *row = tgt + ((size_t)b * T + at) * (size_t)V * Elt<DT>::BYTES;
    chunk_best<DT>(row, V, c, part + (size_t)blockIdx.x * WAVES);
}

template <int DT>
hipError_t tree_by_levels(const Launch &ln, const Workspace &ws, int B, int T, int V, int depth, const char *tgt,
                          const int *tokens, const int *parents, const int *counts, int *acc, int *path, int *out)
{
    const int nch = num_chunks(NV_ARGMAX, DT, V);
    float2 *half[2] = {ws.part, ws.part + (size_t)B * nch * WAVES};
    // the argmax kind is timed from the first depth's start to the last's end
    const bool time = timed(ln, KIND_ARGMAX);
    hipEvent_t first[2 * NUM_KINDS] = {}, last[2 * NUM_KINDS] = {};
    if (time) {
        first[2 * KIND_ARGMAX] = ln.ev[2 * KIND_ARGMAX];
        (depth > 0 ? last : first)[2 * KIND_ARGMAX + 1] = ln.ev[2 * KIND_ARGMAX + 1];
    }
    const Launch plain = {ln.stream, nullptr, 0}, begin = {ln.stream, time ? first : nullptr, ln.mask},
                 finish = {ln.stream, time ? last : nullptr, ln.mask};
    for (int level = 0; level <= depth + 1; ++level) {
        // the last one finishes the walks that went all the way down
        const bool end = level > depth;
        const int groups = end ? 1 : nch;
        const Launch &l = end ? ln : level == 0 ? begin : level == depth ? finish : plain;
        SV_LAUNCH(l, end ? KIND_GREEDY_EMIT : KIND_ARGMAX, k_tree_level<DT>, dim3((unsigned)((size_t)B * groups)),
                  dim3(WG), 0, tgt, tokens, parents, counts, T, V, depth, level, groups, nch, half[(level + 1) & 1],
                  half[level & 1], acc, path, out);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_greedy_tree(const Launch &ln, const Workspace &ws, int cus, int dtype, int B, int T, int V,
                              int depth, const void *tgt, const int32_t *tokens,
                              const int32_t *parents, const int32_t *counts, int32_t *acc_len,
                              int32_t *path, int32_t *out_tokens, unsigned *kinds)
{
    const TreeForm form = tree_form(cus, dtype, B, T, V, depth);
    if (form == TREE_SHORT) {
        const dim3 threads(64 * std::min(T, TREE_WAVES));
        *kinds = 1u << KIND_GREEDY_EMIT;
        if (dtype == 1)
            SV_LAUNCH(ln, KIND_GREEDY_EMIT, k_tree_short<1>, dim3(B), threads, 0, static_cast<const char *>(tgt),
                      tokens, parents, counts, T, V, depth, acc_len, path, out_tokens);
        else
            SV_LAUNCH(ln, KIND_GREEDY_EMIT, k_tree_short<0>, dim3(B), threads, 0, static_cast<const char *>(tgt),
                      tokens, parents, counts, T, V, depth, acc_len, path, out_tokens);
        return hipGetLastError();
    }
    *kinds = 1u << KIND_ARGMAX | 1u << KIND_GREEDY_EMIT;
    if (form == TREE_LEVELS)
        return (dtype == 1 ? tree_by_levels<1> : tree_by_levels<0>)(ln, ws, B, T, V, depth,
                                                                  static_cast<const char *>(tgt), tokens, parents,
                                                                  counts, acc_len, path, out_tokens);
    const int nch = num_chunks(NV_ARGMAX, dtype, V), np = nch * WAVES;
    const dim3 chunks((unsigned)((size_t)B * T * nch));
    if (dtype == 1)
        SV_LAUNCH(ln, KIND_ARGMAX, k_tree_rows<1>, chunks, dim3(WG), 0, static_cast<const char *>(tgt), V, nch, ws.part);
    else
        SV_LAUNCH(ln, KIND_ARGMAX, k_tree_rows<0>, chunks, dim3(WG), 0, static_cast<const char *>(tgt), V, nch, ws.part);
    SV_LAUNCH(ln, KIND_GREEDY_EMIT, k_tree_walk, dim3(B), dim3(64), 0, tokens, parents, counts, T, V, depth, np,
              ws.part, acc_len, path, out_tokens);
    return hipGetLastError();
}

// ------------------------------------------------------------------ the accepted path's tokens

namespace {

constexpr int KEEP_WG = 256;

// A thread has sizeof(V) bytes of a token in one pool and moves them for every node of the path in
// turn, so that a place is read before the thread writes it: places ascend, and a node moves down
// or stays.  Four loads are under way at once: the places that they are stored to are below those
// that later ones read (one at a time: 29 us where it is 18.4 now, 69 MB at 3.8 TB/s).  Few paths are
// bound by the call: 6.5 us.
template <typename V> __global__ __launch_bounds__(KEEP_WG) void k_keep_path(CacheView c, int n, int max_count,
                                                                            int groups, const int *seqs,
                                                                            const int *accepted, const int *path,
                                                                            int *status)
{
    __shared__ int64_t from[MAX_NODES], to[MAX_NODES];
    __shared__ int moves;
    const int i = blockIdx.x / groups, group = blockIdx.x - i * groups, t = threadIdx.x, lane = t & 63;
    const int token = (int)(c.page_bytes / c.page_tokens);
    const int s = seqs ? seqs[i] : i;
    const int acc = accepted[i];
    bool ok = in_range(s, c.num_seqs) && acc >= -1 && acc < max_count;
    if (ok && seqs) {
        bool named = false;
        for (int j = t; j < i; j += KEEP_WG)
            named |= seqs[j] == s;
        ok = !__syncthreads_or(named);
    }
    if (ok) {
        const int had = c.blocks[s], len = c.lengths[s];
        const bool sound = had >= 0 && had <= c.max_blocks && len >= 0 && len <= had * c.page_tokens;
        const int room = sound ? had * c.page_tokens - len : 0;
        const int node = lane <= acc ? path[(size_t)i * max_count + lane] : -1;
        const int before = __shfl_up(node, 1);
        const bool bad = lane <= acc && (lane == 0 ? node != 0 : node <= before || node >= room);
        ok = sound && __ballot(bad) == 0;
        if (ok && t < 64) {
            const int *row = c.tables + (size_t)s * c.max_blocks;
            bool moved = lane > 0 && lane <= acc && node != lane;
            int64_t a = 0, b = 0;
            if (moved) {
                const int pa = row[(len + node) / c.page_tokens], pb = row[(len + lane) / c.page_tokens];
                moved = in_range(pa, c.num_pages) && in_range(pb, c.num_pages);
                a = (int64_t)pa * c.page_bytes + (int64_t)((len + node) % c.page_tokens) * token;
                b = (int64_t)pb * c.page_bytes + (int64_t)((len + lane) % c.page_tokens) * token;
            }
            const uint64_t all = __ballot(moved);
            const int at = __popcll(all & ((1ull << lane) - 1));
            if (moved) {
                from[at] = a;
                to[at] = b;
            }
            if (lane == 0)
                moves = __popcll(all);
        }
    }
    if (status && group == 0 && t == 0)
        status[i] = ok ? 0 : -1;
    if (!ok)
        return;
    __syncthreads();
    const int most = moves, cols = token / (int)sizeof(V);
    for (int64_t x = (int64_t)group * KEEP_WG + t; x < (int64_t)cols * c.num_pools; x += (int64_t)groups * KEEP_WG) {
        const int pool = (int)(x / cols);
        char *p = c.pools[pool] + (x - (int64_t)pool * cols) * (int64_t)sizeof(V);
        for (int j = 0; j < most; j += 4) {
            // four variables: an array of them would live in LDS
            const bool h1 = j + 1 < most, h2 = j + 2 < most, h3 = j + 3 < most;
            V v0 = load_global<V>(p + from[j]), v1 = v0, v2 = v0, v3 = v0;
            if (h1)
                v1 = load_global<V>(p + from[j + 1]);
            if (h2)
                v2 = load_global<V>(p + from[j + 2]);
            if (h3)
                v3 = load_global<V>(p + from[j + 3]);
            store_global<V>(p + to[j], v0);
            if (h1)
                store_global<V>(p + to[j + 1], v1);
            if (h2)
                store_global<V>(p + to[j + 2], v2);
            if (h3)
                store_global<V>(p + to[j + 3], v3);
        }
    }
}

template <typename V> hipError_t keep_with(hipStream_t st, const CacheView &c, int n, int max_count,
                                           const int *seqs, const int *accepted, const int *path, int *status)
{
    const int64_t items = c.page_bytes / c.page_tokens / (int64_t)sizeof(V) * c.num_pools;
    // one item to a thread, as far as a launch holds them
    const int64_t most = std::max<int64_t>(1, (1 << 23) / n);
    const int64_t groups = std::min(std::max<int64_t>(1, (items + KEEP_WG - 1) / KEEP_WG), most);
    k_keep_path<V><<<(unsigned)(groups * n), KEEP_WG, 0, st>>>(c, n, max_count, (int)groups, seqs, accepted,
                                                             path, status);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_keep_path(hipStream_t st, const CacheView &c, int n, int max_count, const int *seqs,
                            const int *accepted, const int *path, int *status)
{
    const int64_t token = c.page_bytes / c.page_tokens;
    if (token % 16 == 0)
        return keep_with<u32x4>(st, c, n, max_count, seqs, accepted, path, status);
    if (token % 4 == 0)
        return keep_with<uint32_t>(st, c, n, max_count, seqs, accepted, path, status);
    return keep_with<uint8_t>(st, c, n, max_count, seqs, accepted, path, status);
}

}  // namespace sv
