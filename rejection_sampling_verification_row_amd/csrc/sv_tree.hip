// Greedy verify of a drafted tree, and the move of its accepted path in a cache (gfx950).
//
// The walk needs the argmax of one row a depth.  All rows at once is one launch that reads
// everything and a launch that walks; depth by depth is a launch for each depth, which reads one row
// of each sequence that is still walking.  In a launch of the latter every workgroup merges its
// sequence's partials of the depth before, finds the next node and reads its chunk of that row, so
// that no workgroup waits for another.
#include <algorithm>
#include <limits.h>

#include "sv_device.h"
#include "sv_internal.h"

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

}  // namespace

hipError_t launch_greedy_tree(const Launch &ln, const Workspace &ws, int dtype, int B, int T, int V,
                              int depth, const void *tgt, const int32_t *tokens,
                              const int32_t *parents, const int32_t *counts, int32_t *acc_len,
                              int32_t *path, int32_t *out_tokens)
{
    const int np = num_chunks(NV_ARGMAX, dtype, V) * WAVES;
    const hipError_t e = launch_argmax_rows(ln, ws, dtype, (size_t)B * T, V, tgt);
    if (e != hipSuccess)
        return e;
    SV_LAUNCH(ln, KIND_GREEDY_EMIT, k_tree_walk, dim3(B), dim3(64), 0, tokens, parents, counts, T, V, depth, np,
              ws.part, acc_len, path, out_tokens);
    return hipGetLastError();
}

// ------------------------------------------------------------------ the accepted path's tokens

namespace {

constexpr int KEEP_WG = 256;
constexpr int KEEP_BATCH = 4;

// A thread has 4 * W bytes of a token in one pool and moves them for every node of the path in
// turn, so that a place is read before the thread writes it: places ascend, and a node moves down
// or stays.  KEEP_BATCH loads are under way at once: the places that a batch writes are below those
// that later ones read.
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
        for (int j = 0; j < most; j += KEEP_BATCH) {
            V v[KEEP_BATCH];
#pragma unroll
            for (int k = 0; k < KEEP_BATCH; ++k)
                if (j + k < most)
                    v[k] = *reinterpret_cast<const V *>(p + from[j + k]);
#pragma unroll
            for (int k = 0; k < KEEP_BATCH; ++k)
                if (j + k < most)
                    *reinterpret_cast<V *>(p + to[j + k]) = v[k];
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
        return keep_with<uint4>(st, c, n, max_count, seqs, accepted, path, status);
    if (token % 4 == 0)
        return keep_with<uint32_t>(st, c, n, max_count, seqs, accepted, path, status);
    return keep_with<uint8_t>(st, c, n, max_count, seqs, accepted, path, status);
}

}  // namespace sv
