// Attention of a verify step's nodes over a paged cache, and the append of their keys and values
// (gfx950).
//
// A row is a query head of a node.  With x_j = scale q . k_j over the tokens j that the node sees (the
// sequence's cached tokens, its ancestors and itself, the last `window` of them) and m = max_j x_j,
//
//     out = sum_j exp(x_j - m) v_j / sum_j exp(x_j - m),    lse = m + log(sum_j exp(x_j - m)).
//
// One pass over the tokens: m is a running maximum, and what was summed under an older one is scaled
// by exp(old - new).  Scores, maxima and sums are fp32, and so is the product with the values, whose
// right side, the weights, is rounded to bfloat16 in bfloat16 pools: a weight is off by at most 2^-8 of
// itself, as the values and the output already are.  (Over whole outputs of random rows the mean square error relative
// to theirs is 2.0e-3 to 2.4e-3, of which the output's own rounding is 1.66e-3; weights in fp32 would take
// matrix instructions at a ninth of the rate, or twice as many.)  exp is computed as a power of 2.
//
// All rows of a key head and an entry read the same keys, so that they are the columns of one matrix:
// S^T = K Q^T, then O^T = V^T P^T.  In the accumulator layout of a 16x16 matrix instruction a lane then
// holds scores of one row, so that a row's maximum and sum stay in the lane but for two exchanges at
// the end, and the weights are, as they lie, the right operand of the second product: the order in
// which a product runs over the tokens is free as long as V^T is read in the same.
//
// Up to 16 rows are bound by memory: k_attend reads keys and values into registers, from where
// they are used once.  More rows in bfloat16 share them: k_attend_wide brings them into LDS.  Which
// form has how many rows, and why, is said at launch_attend.
//
// The lengths are known on the device only.  All tiles of tokens of all entries stand in a row, and
// every workgroup adds the lengths up and takes an equal stretch of it, whatever segments of tokens
// (an entry's, for a key head and a tile of rows) begin or end there.  What a stretch has of a split
// segment is left in the workspace in fp32, and k_attend_join adds the parts in the tokens' order, so
// that results do not depend on which workgroup is done first.
#include <algorithm>
#include <type_traits>

#include "sv_internal.h"
#include "sv_memory.h"

namespace sv {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;
// How far, in powers of 2, scores may exceed the running maximum before k_attend_wide lets it follow: most
// rows' maxima need to follow once.  It weighs against a reference as much above the maximum, so that no
// weight is above 1 and sums pass fp32 only where values do; weights of 2^-8 where 1 would stand lose nothing.
// (512 rows of heads of 128 505 -> 510 us; the others alike.)
constexpr float LAG = 8.0f;
// Raw scores from FAR / c1 on would pass fp32 once they are in powers of 2; weights are then formed from
// differences of raw scores.  What waves and parts hand on of their maxima is a quarter, which any score's is in fp32.
constexpr float FAR = 3e38f, QUARTER = 0.25f;

__device__ inline bool in_range(int i, int n) { return (unsigned)i < (unsigned)n; }

// a value that all lanes have
__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline double uniform(double v)
{
    return __hiloint2double(uniform(__double2hiint(v)), uniform(__double2loint(v)));
}

// The same value, of which the compiler knows nothing: what is computed from it stays where it is
// written, and takes no registers elsewhere.
__device__ inline int afresh(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

__device__ inline int divide(int j, const FastDiv &f)
{
    return f.s < 0 ? j : (int)(__umulhi((uint32_t)j, f.m) >> f.s);
}

// ------------------------------------------------------------------ entries and nodes

struct Entry {
    int seq, start, count, len;      // count < 0: refused
};

__device__ inline Entry load_entry(const CacheView &c, const NodesView &nv, int i)
{
    Entry e = {-1, 0, -1, 0};
    const int s = nv.seqs ? nv.seqs[i] : i;
    if (!in_range(s, c.num_seqs))
        return e;
    const int64_t start = nv.starts ? nv.starts[i] : (int64_t)i * nv.max_count;
    const int cnt = nv.counts ? nv.counts[i] : nv.max_count;
    const int had = c.blocks[s], len = c.lengths[s];
    if (had < 0 || had > c.max_blocks || len < 0 || len > had * c.page_tokens)
        return e;
    if (cnt < 0 || cnt > nv.max_count || cnt > had * c.page_tokens - len || start < 0 ||
        start + cnt > nv.rows)
        return e;
    e.seq = s;
    e.start = (int)start;
    e.count = cnt;
    e.len = len;
    return e;
}

// Lane t's node: its ancestors and itself as bits, and its depth; false when a parent is not below
// its child.  Of `window` depths only, if that is above 0.  Whole waves call it.  Ancestors are
// joined over 1, 2, 4, ... 32 steps at a time.
__device__ inline bool lane_node(const int *parents, int count, int window, uint64_t &seen, int &depth)
{
    const int t = threadIdx.x & 63;
    int up = t < count ? t - 1 : -1;
    if (parents && t > 0 && t < count)
        up = parents[t];
    const bool bad = t > 0 && t < count && (up < 0 || up >= t);
    if (__ballot(bad) != 0)
        return false;
    seen = 1ull << t;
#pragma unroll
    for (int k = 0; k < 6; ++k) {
        const uint64_t more = __shfl((unsigned long long)seen, max(up, 0));
        const int far = __shfl(up, max(up, 0));
        if (up >= 0) {
            seen |= more;
            up = far;
        }
    }
    depth = __popcll(seen) - 1;
    if (window > 0 && window < MAX_NODES) {
        uint64_t near = 0;
        for (int a = 0; a < count; ++a)
            if (depth - __shfl(depth, a) < window)
                near |= 1ull << a;
        seen &= near;
    }
    return true;
}

// ------------------------------------------------------------------ attention

struct AttnArgs {
    CacheView c;
    AttnShape a;
    NodesView nv;
    int key_pool, value_pool;
    float c1;            // |scale| log2(e), 1 for scale 0
    float far;           // FAR / c1
    float q_sign;        // the queries' factor: scale's sign
    int window;
    const char *q;
    int64_t q_stride;    // bytes
    char *out;
    int64_t out_stride;  // bytes
    float *lse;
    int *status;
    int units;           // workgroups that fill the chip
};

// The arguments read again: what comes from them is not kept in registers, or computed ahead, over a
// whole kernel.
__device__ inline AttnArgs args_afresh()
{
    auto p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    AttnArgs a;
    __builtin_memcpy(&a, p, sizeof a);
    return a;
}

// Inclusive sum over the workgroup's threads; *all is the whole.  Counts of tiles are doubles: exact
// up to 2^53, and sums and quotients of them take few instructions.
template <int WG_SIZE> __device__ inline double block_scan(double v, double *lds, double *all)
{
    const int w = threadIdx.x >> 6;
    const double inc = wave_incl_scan(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 63)
        lds[w] = inc;
    __syncthreads();
    double before = 0.0, sum = 0.0;
#pragma unroll
    for (int i = 0; i < WG_SIZE / 64; ++i) {
        before += i < w ? lds[i] : 0.0;
        sum += lds[i];
    }
    *all = uniform(sum);
    return before + inc;
}

// An entry's work: segments (key heads times tiles of rows) and tiles of KT tokens from `low` on.  A
// segment counts AHEAD tiles more, which stand before its own: what it takes to begin and to end one
// (queries, first loads, the waves' sums).  Without, stretches of many short segments were the last to end.
// 64 sequences of 300 to 8200 tokens in k_attend_wide, AHEAD of 0, 768 and 1536 tokens: 32 rows 236, 210
// and 216 us, 128 rows 375, 270 and 274 us; in k_attend, 24 float32 sequences in a window of 2000, 0, 6 and
// 20 tiles: 72, 59 and 61 us.
struct Work {
    int tiles_of_rows, segments, low, tiles, counted;
    __device__ double all() const { return (double)segments * (double)counted; }
};

template <int KT, int AHEAD> __device__ inline Work entry_work(const AttnArgs &a, const Entry &e, int rows_per_tile)
{
    Work w = {0, 0, 0, 0, 0};
    if (e.count <= 0)
        return w;
    w.tiles_of_rows = (e.count * a.a.group + rows_per_tile - 1) / rows_per_tile;
    w.segments = w.tiles_of_rows * a.a.kv_heads;
    // the root is the first to see least far back
    w.low = a.window > 0 ? max(e.len - a.window + 1, 0) / KT : 0;
    w.tiles = (int)(((unsigned)e.len + e.count + KT - 1) / KT) - w.low;
    w.counted = w.tiles + AHEAD;
    return w;
}

// All tiles stand in a row, entry by entry and in an entry segment by segment, and every workgroup
// takes the same number of them.  What it works on, in LDS, so that it takes no registers while it
// works: tiles t0 .. t1 of a segment's tokens, then from `at` on.
struct Job {
    double at, end;                      // its stretch of all tiles, what is left of it
    double base;                         // the entry's first tile among all
    int mine;                            // the stretch's number; < 0: none, or nothing left
    int entry;
    Entry e;
    int head, mt, t0, t1;
    int opens;                           // this is the entry's first tile
    int whole;                           // all of the segment; else the sums go to this slot of the kept ones:
    int slot;
};

// This workgroup's stretch and the entry that it begins in.  Workgroup 0 also leaves the plan for the
// join, and the status of entries that have no work.  False: there is no stretch for it.
template <int WG_SIZE, int KT, int AHEAD>
__device__ bool find_stretch(const AttnArgs &a, int rows_per_tile, int least, Job &job)
{
    __shared__ double lds[WG_SIZE / 64];
    const int n = a.nv.n, t = threadIdx.x;
    Entry e = {-1, 0, -1, 0};
    if (t < n)
        e = load_entry(a.c, a.nv, t);
    Work w = entry_work<KT, AHEAD>(a, e, rows_per_tile);
    double sum, first = block_scan<WG_SIZE>(w.all(), lds, &sum) - w.all();
    const double part = sum;             // of the first WG_SIZE entries
    for (int i0 = WG_SIZE; i0 < n; i0 += WG_SIZE) {
        const int i = i0 + t;
        double more = 0.0, all;
        if (i < n)
            more = entry_work<KT, AHEAD>(a, load_entry(a.c, a.nv, i), rows_per_tile).all();
        block_scan<WG_SIZE>(more, lds, &all);
        sum += all;
    }
    const double share = fmax(floor(sum / a.units) + 1.0, (double)least);
    // neighbours, which read the same tokens, on one of the 8 dies, to which workgroups go in turn
    const int active = (int)ceil(sum / share), each = (active + 7) / 8;
    int mine = (int)(blockIdx.x & 7) * each + (int)(blockIdx.x >> 3);
    const double at = mine * share;
    if ((int)(blockIdx.x >> 3) >= each || at >= sum)
        mine = -1;
    if (mine < 0 && blockIdx.x != 0)
        return false;
    double base = part;
    for (int i0 = 0; i0 < n; i0 += WG_SIZE) {
        const int i = i0 + t;
        if (i0 > 0) {
            e = {-1, 0, -1, 0};
            if (i < n)
                e = load_entry(a.c, a.nv, i);
            w = entry_work<KT, AHEAD>(a, e, rows_per_tile);
            double all;
            first = base + block_scan<WG_SIZE>(w.all(), lds, &all) - w.all();
            base += all;
        }
        if (mine >= 0 && at >= first && at < first + w.all()) {
            job.at = at;
            job.end = fmin(at + share, sum);
            job.base = first;
            job.mine = mine;
            job.entry = i;
            job.e = e;
        }
        if (blockIdx.x == 0 && i < n) {
            a.a.plan[i] = {first, w.counted, w.tiles, w.tiles_of_rows, e.start, max(e.count, 0)};
            if (a.status && w.segments == 0)
                a.status[i] = e.count < 0 ? -1 : 0;
        }
    }
    if (blockIdx.x == 0 && t == 0)
        *a.a.share = share;
    __syncthreads();
    return mine >= 0;
}

// The next job of the stretch, found by the first wave; false at its end.
template <int KT, int AHEAD> __device__ inline bool next_job(const AttnArgs &a, int rows_per_tile, Job &job)
{
    if (threadIdx.x < 64) {
        double at = uniform(job.at), base = uniform(job.base);
        const double end = uniform(job.end);
        int entry = uniform(job.entry), t0 = 0, t1 = 0;
        double segment = 0.0;
        Entry e = {uniform(job.e.seq), uniform(job.e.start), uniform(job.e.count), uniform(job.e.len)};
        Work w = entry_work<KT, AHEAD>(a, e, rows_per_tile);
        // what ends before a segment's own tiles is no job
        while (at < end && t0 == t1) {
            // `entry` stays below n whatever other work does to the lengths meanwhile
            while (at >= base + w.all() && entry + 1 < a.nv.n) {
                base += w.all();
                e = load_entry(a.c, a.nv, ++entry);
                w = entry_work<KT, AHEAD>(a, e, rows_per_tile);
            }
            segment = floor((at - base) / w.counted);
            const int off = (int)(at - base - segment * w.counted);
            const int take = max((int)fmin((double)(w.counted - off), end - at), 1);
            at += take;
            t0 = max(off - AHEAD, 0);
            t1 = max(off + take - AHEAD, 0);
        }
        if (threadIdx.x == 0) {
            if (t0 == t1) {
                job.mine = -1;
            } else {
                job.at = at;
                job.base = base;
                job.entry = entry;
                job.e = e;
                job.head = (int)segment / w.tiles_of_rows;
                job.mt = (int)segment - job.head * w.tiles_of_rows;
                job.t0 = w.low + t0;
                job.t1 = w.low + t1;
                job.opens = segment == 0.0 && t0 == 0;
                job.whole = t0 == 0 && t1 == w.tiles;
                job.slot = 2 * job.mine + (t0 == 0);
            }
        }
    }
    __syncthreads();
    return uniform(job.mine) >= 0;
}

// Whether the parents of the job's entry are sound, and if so what a lane's node sees; the workgroup
// that has the entry's first tile says it.
__device__ inline bool open_job(const AttnArgs &a, const Job &job, uint64_t &seen, int &depth)
{
    const int start = uniform(job.e.start), count = uniform(job.e.count);
    const bool ok = lane_node(a.nv.parents ? a.nv.parents + start : nullptr, count, a.window, seen, depth);
    if (uniform(job.opens) && threadIdx.x == 0) {
        a.a.sound[job.entry] = ok;
        if (a.status)
            a.status[job.entry] = ok ? 0 : -1;
    }
    return ok;
}

template <int DT> struct Tile;
template <> struct Tile<1> {
    static constexpr int ES = 2, KT = 32;     // bytes of an element, tokens of a tile
    typedef bf16x8 vec;
};
template <> struct Tile<0> {
    static constexpr int ES = 4, KT = 16;
    typedef f32x4 vec;
};

template <int BYTES> struct Chunk;
template <> struct Chunk<16> { typedef u32x4 type; };
template <> struct Chunk<8> { typedef u32x2 type; };

// any element of a word (two bfloat16, or a float) infinite or NaN
template <int DT> __device__ inline bool odd_word(uint32_t w)
{
    if constexpr (DT == 1)
        return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
    else
        return (w & 0x7f800000u) == 0x7f800000u;
}

__device__ inline float row_max(float v)
{
    v = fmaxf(v, xch<4>(v));
    return fmaxf(v, xch<5>(v));
}
__device__ inline float row_sum(float v)
{
    v += xch<4>(v);
    return v + xch<5>(v);
}

// What stands for elements past a head's end (head_dim below a kernel's size): the queries are 0
// there, and so must the keys be, whatever follows them in memory.
__device__ const uint4 past_the_head = {0, 0, 0, 0};

// A wave's R tiles of rows from `first` on, with their queries as right operands.  What a row sees and
// from which token on go to LDS, the least token that all see is returned.
template <int DT, int KS, int R>
__device__ inline int load_rows(const AttnArgs &a, const Job &job, uint64_t lane_seen, int lane_depth, int first,
                                uint64_t *seen, int *low, typename Tile<DT>::vec (&q)[R][KS])
{
    constexpr int ES = Tile<DT>::ES;
    const int col = threadIdx.x & 15, grp = threadIdx.x >> 4 & 3, D = a.a.head_dim, G = a.a.group;
    const int start = uniform(job.e.start), len = uniform(job.e.len), rows = uniform(job.e.count) * G;
    const char *base = a.q + (int64_t)start * a.q_stride + (int64_t)uniform(job.head) * G * D * ES;
    int most = 0;
    u32x4 v[R][KS];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int row = first + r * 16 + col;
        const int node = row < rows ? divide(row, a.a.by_group) : 0;
        const uint64_t sees = __shfl((unsigned long long)lane_seen, node);
        const int depth = __shfl(lane_depth, node), from = a.window > 0 ? max(len - a.window + 1 + depth, 0) : 0;
        most = max(most, from);
        if (grp == 0) {
            seen[r * 16 + col] = sees;
            low[r * 16 + col] = from;
        }
        const char *qp = base + node * a.q_stride + (row - node * G) * D * ES;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = (s * 64 + grp * 16) / ES;
            v[r][s] = u32x4{0, 0, 0, 0};
            if (row < rows && d < D)
                v[r][s] = load_global<u32x4_any>(qp + d * ES);
        }
    }
    // scale's sign
    const uint32_t keep = a.q_sign == 0.0f ? 0u : ~0u;
    const uint32_t flip = a.q_sign < 0.0f ? (DT == 1 ? 0x80008000u : 0x80000000u) : 0u;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int s = 0; s < KS; ++s)
            q[r][s] = __builtin_bit_cast(typename Tile<DT>::vec, (v[r][s] & keep) ^ flip);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1)
        most = max(most, __shfl_xor(most, o));
    return uniform(most);
}

// Which of the 32 tokens from j0 on a row sees, as bits.
__device__ inline uint32_t visible(int len, int low, uint64_t seen, int j0, uint32_t lost)
{
    const int back = len - j0, from = low - j0;
    uint32_t v = back >= 32 ? ~0u : back > 0 ? (1u << back) - 1 : 0;
    v = from >= 32 ? 0 : from > 0 ? v & (~0u << from) : v;
    if (back <= 0)
        v |= back > -64 ? (uint32_t)(seen >> -back) : 0;
    else if (back < 32)
        v |= (uint32_t)seen << back;
    return v & ~lost;
}

template <int SUB> __device__ inline float tile_max(const f32x4 (&s)[SUB])
{
    float top = s[0][0];
#pragma unroll
    for (int x = 0; x < SUB; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            top = fmaxf(top, s[x][i]);
    return top;
}

// The running maxima m (of raw scores) follow a tile's; what was summed before is scaled.
template <int SUB, int NT, int R>
__device__ inline void follow(const f32x4 (&s)[R][SUB], f32x4 (&o)[R][NT], float (&m)[R], float (&l)[R], float c1)
{
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float was = m[r];
        m[r] = fmaxf(was, row_max(tile_max<SUB>(s[r])));
        const float f = m[r] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((was - m[r]) * c1);
        l[r] *= f;
#pragma unroll
        for (int i = 0; i < NT; ++i)
            o[r][i] *= f;
    }
}

// Whether a maximum is FAR, though not of nothing.
template <int R> __device__ inline bool any_far(const float (&m)[R], float far)
{
    bool any = false;
#pragma unroll
    for (int r = 0; r < R; ++r)
        any |= !(fabsf(m[r]) < far) && m[r] != -INFINITY;
    return __ballot(any) != 0;
}

// Scores of a tile become weights against what is `above` the maxima in powers of 2, and are summed.  DIFF: maxima
// may be FAR; else rows of such have no scores here but -inf and NaN.
template <bool DIFF, int SUB, int R>
__device__ inline void weigh(f32x4 (&s)[R][SUB], const float (&m)[R], float (&l)[R], float c1, float far,
                             float above)
{
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float ref = DIFF ? (m[r] == -INFINITY ? 0.0f : m[r]) : fabsf(m[r]) < far ? m[r] * c1 + above : 0.0f;
        float sum[SUB];
#pragma unroll
        for (int x = 0; x < SUB; ++x) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s[r][x][i] = __builtin_amdgcn_exp2f(DIFF ? __builtin_fmaf(s[r][x][i] - ref, c1, -above)
                                                         : __builtin_fmaf(s[r][x][i], c1, -ref));
            sum[x] = (s[r][x][0] + s[r][x][1]) + (s[r][x][2] + s[r][x][3]);
        }
        l[r] += SUB == 2 ? sum[0] + sum[SUB - 1] : sum[0];
    }
}

// What sums under a maximum count under a higher one, of quarters; the log of a whole sum.
__device__ inline float scale_down(float was, float top)
{
    return was == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f((was - top) / QUARTER);
}
__device__ inline float log_sum(float top, float z)
{
    const float whole = top / QUARTER;
    if (fabsf(whole) == INFINITY && fabsf(top) < INFINITY)
        return top * (LN2 / QUARTER);          // beside which log z is nothing
    return z == 0.0f ? -INFINITY : (whole + log2f(z)) * LN2;
}

// The sums of `waves` waves over a tile of rows, joined, to the output or to the kept ones: row i at
// o[wave * wave_step + i], its maximum (a quarter) and sum at ml of the same index.
template <int DT, int WG_SIZE, int PITCH>
__device__ inline void finish(const AttnArgs &a, const Job &j, int rows_per_tile, const float (*o)[PITCH],
                              const float2 *ml, int waves, int wave_step)
{
    constexpr int ES = Tile<DT>::ES;
    const int D = a.a.head_dim, G = a.a.group, first = j.mt * rows_per_tile;
    const int rows = min(j.e.count * G - first, rows_per_tile);
    for (int i = threadIdx.x; i < rows * (D / 4); i += WG_SIZE) {
        const int row = i / (D / 4), d = (i - row * (D / 4)) * 4;
        float top = -INFINITY;
        for (int k = 0; k < waves; ++k)
            top = fmaxf(top, ml[k * wave_step + row].x);
        float z = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < waves; ++k) {
            const float2 p = ml[k * wave_step + row];
            const float f = scale_down(p.x, top);
            z += f * p.y;
            const float4 v = *reinterpret_cast<const float4 *>(&o[k * wave_step + row][d]);
            acc[0] += f * v.x;
            acc[1] += f * v.y;
            acc[2] += f * v.z;
            acc[3] += f * v.w;
        }
        if (!j.whole) {
            const int64_t at = (int64_t)j.slot * rows_per_tile + row;
            *reinterpret_cast<float4 *>(a.a.part_o + at * D + d) = make_float4(acc[0], acc[1], acc[2], acc[3]);
            if (d == 0)
                a.a.part_ml[at] = make_float2(top, z);
            continue;
        }
        const int gr = first + row, node = divide(gr, a.a.by_group), qh = j.head * G + gr - node * G;
        char *to = a.out + (int64_t)(j.e.start + node) * a.out_stride + ((int64_t)qh * D + d) * ES;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float v = z == 0.0f ? 0.0f : acc[x] / z;
            if constexpr (DT == 1)
                reinterpret_cast<__bf16 *>(to)[x] = (__bf16)v;
            else
                reinterpret_cast<float *>(to)[x] = v;
        }
        if (a.lse && d == 0)
            a.lse[(int64_t)(j.e.start + node) * a.a.q_heads + qh] = log_sum(top, z);
    }
}

// Few rows: each of four waves has tiles of tokens of its own, whose keys and values it loads into
// registers a tile ahead, keys straight in the left operand's layout, values with lanes along the
// head, of which for 16-bit values pairs of tokens are joined by byte permutes.  Waves meet only at a
// segment's end.
//
// Bound by memory, for one sequence by the way to the first load: 64 sequences of 300 to 8200 tokens,
// 8 key heads of 128 in bfloat16, 4 rows each: 211 us, 5.3 TB/s; float32, 4 key heads of 128: 193 us,
// 5.8 TB/s; one sequence of 1000 tokens: 9 us and 4 us of the join.  Of those 9 us the loop is 2; what comes
// before it is short because it is not kept in registers from one job to the next (args_afresh: 14.5 ->
// 12.9 us) and because stretches are counted in doubles (64-bit integer division: 15.4 -> 14.6 us).
//
// DP: head_dim or more; VW: elements of a value row that a lane loads at once, 16 lanes side by
// side; R: tiles of 16 rows.  Left operands of the products: row lane % 16, 16 bytes (4 for float32)
// of the axis summed over to each of the four groups lane / 16; right ones likewise with columns;
// results: column lane % 16, rows 4 (lane / 16) + r.
template <int DT, int DP, int VW, int R, int OCC>
__global__ __launch_bounds__(ATTN_WG, OCC) void k_attend(AttnArgs args)
{
    typedef Tile<DT> TL;
    constexpr int ES = TL::ES, KT = TL::KT, SUB = KT / 16, KPL = KT / 4;
    constexpr int KS = DP * ES / 64;              // 16-byte pieces of a key row to a lane
    constexpr int NB = DP / (16 * VW);            // pieces of a value row to a lane
    constexpr int NT = DP / 16;
    constexpr int ROWS = 16 * R, PITCH = DP + 4, AHEAD = 6;
    typedef typename Chunk<VW * ES>::type vchunk;

    __shared__ float s_o[4 * ROWS][PITCH];
    __shared__ float2 s_ml[4 * ROWS];
    __shared__ int64_t s_off[4][2][KT];
    __shared__ uint64_t s_seen[ROWS];
    __shared__ int s_low[ROWS];
    __shared__ Job job;

    if (!find_stretch<ATTN_WG, KT, AHEAD>(args, ROWS, 128 / KT, job))
        return;
    while (next_job<KT, AHEAD>(args_afresh(), ROWS, job)) {
        const AttnArgs a = args_afresh();
        const int thread = afresh(threadIdx.x), lane = thread & 63, w = uniform(thread >> 6);
        const int col = lane & 15, grp = lane >> 4;
        uint64_t lane_seen;
        int lane_depth;
        const bool ok = open_job(a, job, lane_seen, lane_depth);
        const int D = a.a.head_dim, len = uniform(job.e.len), total = len + uniform(job.e.count);
        const int t0 = uniform(job.t0), t1 = uniform(job.t1), head = uniform(job.head);
        typename TL::vec q[R][KS];
        // all waves write the same rows
        const int low_most =
            ok ? load_rows<DT, KS, R>(a, job, lane_seen, lane_depth, uniform(job.mt) * ROWS, s_seen, s_low, q) : 0;
        if (!ok) {
            __syncthreads();
            continue;
        }

        const int *table = a.c.tables + (size_t)uniform(job.e.seq) * a.c.max_blocks;
        const int64_t row_bytes = (int64_t)a.a.kv_heads * D * ES;
        const char *kp = a.c.pools[a.key_pool] + (int64_t)head * D * ES;
        const char *vp = a.c.pools[a.value_pool] + (int64_t)head * D * ES;
        const char *zeros = reinterpret_cast<const char *>(&past_the_head);

        // a tile's page ids, one token to a lane, then the tokens' places; bits of what has no place
        auto page_of = [&](int tile) {
            const int j = (int)min((unsigned)tile * KT + (lane & (KT - 1)), (unsigned)total - 1);
            return load_global<int>(table + divide(j, a.a.by_page));
        };
        auto put_places = [&](int tile, int pg, int buf) {
            const int j = (int)min((unsigned)tile * KT + (lane & (KT - 1)), (unsigned)total - 1);
            const int b = divide(j, a.a.by_page);
            const bool good = in_range(pg, a.c.num_pages);
            const int64_t at = (int64_t)(good ? pg : 0) * a.c.page_tokens + (j - b * a.c.page_tokens);
            if (lane < KT)
                s_off[w][buf][lane] = at * row_bytes;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
            return (uint32_t)(__ballot(!good) & ((1ull << KT) - 1));
        };

        u32x4 kr[SUB][KS];
        vchunk vr[KPL][NB];
        auto load_keys = [&](int buf) {
#pragma unroll
            for (int s = 0; s < SUB; ++s) {
                const char *p = kp + s_off[w][buf][s * 16 + col];
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const int b = k * 64 + grp * 16;
                    kr[s][k] = load_once<u32x4>(b < D * ES ? p + b : zeros);
                }
            }
        };
        auto load_values = [&](int buf) {
#pragma unroll
            for (int k = 0; k < KPL; ++k) {
                const char *p = vp + s_off[w][buf][(k / 4) * 16 + grp * 4 + (k & 3)];
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int at = (b * 16 + col) * VW * ES;
                    vr[k][b] = load_once<vchunk>(p + (at < D * ES ? at : 0));
                }
            }
        };

        f32x4 o[R][NT];
        float m[R], l[R];                    // maximum of the raw scores, this lane's part of the sum
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                o[r][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }

        bool far = false;
        int t = t0 + w, buf = 0, next_page = 0;
        const int last = t1 - 1 - (t1 - 1 - t & 3);          // this wave's last tile
        uint32_t lost = 0;
        if (t < t1) {
            lost = put_places(t, page_of(t), 0);
            load_keys(0);
            load_values(0);
            next_page = page_of(min(t + 4, last));
        }
        for (; t < t1; t += 4, buf ^= 1) {
            f32x4 s[R][SUB];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int x = 0; x < SUB; ++x) {
                    s[r][x] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
                        const typename TL::vec kv = __builtin_bit_cast(typename TL::vec, kr[x][k]);
                        if constexpr (DT == 1) {
                            s[r][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kv, q[r][k], s[r][x], 0, 0, 0);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                s[r][x] = __builtin_amdgcn_mfma_f32_16x16x4f32(kv[i], q[r][k][i], s[r][x], 0, 0, 0);
                        }
                    }
                }
            // the next tile's loads are made in any case (the last tile's again): a branch around them
            // would let every wait for older ones wait for all
            const uint32_t next_lost = put_places(min(t + 4, last), next_page, buf ^ 1);
            next_page = page_of(min(t + 8, last));
            load_keys(buf ^ 1);
            const unsigned j0 = (unsigned)t * KT;
            const bool masked = j0 + KT > (unsigned)len || lost != 0 || (int)j0 < low_most;
            uint32_t vis[R];                 // the tile's tokens that a row sees
            if (masked) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    vis[r] = visible(len, s_low[r * 16 + col], s_seen[r * 16 + col], (int)j0, lost);
#pragma unroll
                    for (int x = 0; x < SUB; ++x)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s[r][x][i] = vis[r] >> (grp * 4) & (1u << (x * 16 + i)) ? s[r][x][i] : -INFINITY;
                }
            }
            bool grew = false;
#pragma unroll
            for (int r = 0; r < R; ++r)
                grew |= tile_max<SUB>(s[r]) > m[r];
            if (__ballot(grew) != 0) {
                follow<SUB, NT, R>(s, o, m, l, a.c1);
                far = any_far<R>(m, a.far);
            }
            if (far)
                weigh<true, SUB, R>(s, m, l, a.c1, a.far, 0.0f);
            else
                weigh<false, SUB, R>(s, m, l, a.c1, a.far, 0.0f);
            if (masked) {
                // What a row does not see may be anything: rows of values with an infinity or a NaN are left
                // out of the product and added to the rows that see them, one by one.
                uint32_t odd = 0;
#pragma unroll
                for (int k = 0; k < KPL; ++k) {
                    bool mine = false;
#pragma unroll
                    for (int x = 0; x < NB; ++x)
#pragma unroll
                        for (int i = 0; i < VW * ES / 4; ++i)
                            mine |= odd_word<DT>(vr[k][x][i]);
                    const uint64_t all = __ballot(mine);
                    if (all == 0)
                        continue;
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        odd |= all >> (g * 16) & 0xffff ? 1u << ((k / 4) * 16 + g * 4 + (k & 3)) : 0;
                    if (all >> (grp * 16) & 0xffff)
#pragma unroll
                        for (int x = 0; x < NB; ++x)
                            vr[k][x] = vchunk{};
                }
#pragma unroll 1
                for (; odd != 0; odd &= odd - 1) {
                    const int key = __builtin_ctz(odd), g4 = afresh(grp * 4);
                    const char *p = vp + s_off[w][buf][key];
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float pr = 0.0f;
#pragma unroll
                        for (int x = 0; x < SUB; ++x)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                pr = key / 16 == x && (key & 3) == i ? s[r][x][i] : pr;
                        pr = __shfl(pr, (key >> 2 & 3) * 16 + col);
                        const bool sees = vis[r] >> key & 1;
#pragma unroll
                        for (int x = 0; x < NT; ++x)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                // one after another: all at once would take more registers than there are
                                __builtin_amdgcn_sched_barrier(0);
                                const int d = (x / VW) * 16 * VW + (g4 + i) * VW + x % VW;
                                const char *at = p + (d < D ? d : 0) * ES;
                                float v;
                                if constexpr (DT == 1)
                                    v = __uint_as_float((uint32_t)load_global<uint16_t>(at) << 16);
                                else
                                    v = load_global<float>(at);
                                o[r][x][i] = sees ? o[r][x][i] + pr * v : o[r][x][i];
                            }
                    }
                }
            }
            if constexpr (DT == 1) {
                bf16x8 p[R];
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        p[r][i] = (__bf16)s[r][i / 4][i & 3];
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int x = 0; x < VW; ++x) {
                        uint32_t u[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            u[i] = __builtin_amdgcn_perm(vr[2 * i + 1][b][x / 2], vr[2 * i][b][x / 2],
                                                         x & 1 ? 0x07060302u : 0x05040100u);
                        const bf16x8 vt = __builtin_bit_cast(bf16x8, make_uint4(u[0], u[1], u[2], u[3]));
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            o[r][b * VW + x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, p[r], o[r][b * VW + x],
                                                                                       0, 0, 0);
                    }
            } else {
#pragma unroll
                for (int k = 0; k < KPL; ++k)
#pragma unroll
                    for (int b = 0; b < NB; ++b)
#pragma unroll
                        for (int x = 0; x < VW; ++x)
#pragma unroll
                            for (int r = 0; r < R; ++r)
                                o[r][b * VW + x] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                    __uint_as_float(vr[k][b][x]), s[r][0][k], o[r][b * VW + x], 0, 0, 0);
            }
            load_values(buf ^ 1);
            lost = next_lost;
        }

#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float sum = row_sum(l[r]);
            const int at = w * ROWS + r * 16 + col;
            if (grp == 0)
                s_ml[at] = make_float2(m[r] == -INFINITY ? -INFINITY : m[r] * (a.c1 * QUARTER), sum);
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int x = 0; x < VW; ++x)
                        s_o[at][b * 16 * VW + (grp * 4 + i) * VW + x] = o[r][b * VW + x][i];
        }
        __syncthreads();
        finish<DT, ATTN_WG, PITCH>(a, job, ROWS, s_o, s_ml, 4, ROWS);
        __syncthreads();
    }
}

// The order of a row's 16-byte pieces in LDS: piece p of row r is at p ^ order(r).  Keys: 8 rows'
// equal pieces in different banks; values: 4 rows' equal pairs of pieces.  (64 banks of 4 bytes: rows
// of 128 bytes come in pairs.)
template <int DP> __device__ inline int key_order(int row)
{
    return DP == 64 ? row >> 1 & 7 : row & 15;
}
template <int DP> __device__ inline int value_order(int row)
{
    return DP == 64 ? (row >> 1 & 3) * 2 : (row & 7) * 2;
}

// A load of 16 (4) bytes a lane from memory to LDS, at `to` plus the lane's place; a wave's `to` is
// uniform.  Nothing waits for it but what says so: the compiler, which cannot tell the stages
// apart, would let every read of LDS wait for all of them.
__device__ inline uint32_t lds_address(const void *p)
{
    return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void *)p;
}
// ONCE: no other workgroup reads the same (it need not stay in the caches; attend over 250001 tokens
// 202 -> 184 us).
template <bool ONCE> __device__ inline void load_to_lds16(const char *from, uint32_t to)
{
    if constexpr (ONCE)
        asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" ::"v"(from), "{m0}"(to) : "memory");
    else
        asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(from), "{m0}"(to) : "memory");
}
__device__ inline void load_to_lds4(const void *from, uint32_t to)
{
    asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(from), "{m0}"(to) : "memory");
}

// More rows, bfloat16: eight waves, WR of them side by side over the rows (16 R each) and 8 / WR
// over the tokens, share what a stage of tokens brings from memory straight into LDS, DEPTH stages
// ahead.  KB: blocks of 32 tokens that a wave has in a stage.
//
// LDS holds a token's row of a stage in 16-byte pieces in an order of the row's own, so that 16
// lanes that read the same piece of 16 rows (keys), or 32 bytes of 4 rows (values, which the LDS
// transposes on the way), touch all banks alike: 0.07% of the LDS's active cycles are conflicts.
//
// A block of 32 rows and 32 tokens of heads of 128 is 32 matrix instructions (512 cycles) and some
// 120 others with 16 exponentials (about 630 cycles), which overlap only if the two waves of a SIMD do
// different things.  So with four stages the upper half of the waves meets the stage's barrier between
// its scores and its weights, when the lower half begins with scores, and matrix instructions have
// priority (531 -> 520 us): 16 sequences of 64 nodes, 64 query and 8 key heads, 8000 to 16000 tokens: 510 us,
// 726 TFLOP/s, where a large library product reaches 1352 TFLOP/s.  The matrix units are busy 36% of the time;
// waves wait for barriers and LDS 29% of theirs and for their turn to issue 27%.  Not kept: the next block's
// keys read, or its scores computed, before the weights of this one (no registers are left, 2 times slower).
//
// Fewer rows are bound by memory: 64 sequences of 300 to 8200 tokens with 8 key heads of 128: 32 rows
// 210 us (5.35 TB/s), 64 rows 226 us, 128 rows 270 us.
template <int DP, int R, int WR, int KB, int STAGES>
__global__ __launch_bounds__(ATTN_WIDE_WG, 1) void k_attend_wide(AttnArgs a)
{
    constexpr int WAVES8 = ATTN_WIDE_WG / 64, KG = WAVES8 / WR, TK = KG * KB * 32;
    constexpr int KS = DP / 32, NT = DP / 16, PIECES = DP / 8, ROW = DP * 2;
    constexpr bool SHIFT = STAGES == 4;
    constexpr int ROWS = 16 * R * WR, PITCH = DP + 4, DEPTH = SHIFT ? STAGES - 2 : STAGES - 1;
    constexpr int HALF = TK * ROW, LOADS = HALF / 1024 / WAVES8;      // bytes of keys in a stage; a wave's loads
    constexpr int PAGE_AHEAD = 2 * DEPTH + 1, AHEAD = 768 / TK;
    constexpr int EARLY = NT < 8 ? NT : 8;        // pieces of values read before the weights are there
    static_assert(LOADS * 1024 * WAVES8 == HALF && DEPTH <= 3 && TK <= ATTN_WIDE_WG, "whole loads, rings of 4 stages");
    constexpr int MERGE = WAVES8 * 16 * R * PITCH * 4;
    __shared__ __attribute__((aligned(1024))) char mem[MERGE > STAGES * 2 * HALF ? MERGE : STAGES * 2 * HALF];
    __shared__ float2 s_ml[WAVES8 * 16 * R];
    __shared__ int64_t s_off[4][TK];
    __shared__ int s_page[4][TK < 64 ? 64 : TK];
    __shared__ uint32_t s_lost[8][TK / 32];
    __shared__ uint64_t s_seen[ROWS];
    __shared__ int s_low[ROWS];
    __shared__ Job job;

    const int t = threadIdx.x, lane = t & 63, w = uniform(t >> 6), col = lane & 15, grp = lane >> 4;
    const int rw = w % WR, kg = w / WR;
    if (!find_stretch<ATTN_WIDE_WG, TK, AHEAD>(a, ROWS, 1, job))
        return;
    while (next_job<TK, AHEAD>(a, ROWS, job)) {
        uint64_t lane_seen;
        int lane_depth;
        const bool ok = open_job(a, job, lane_seen, lane_depth);
        if (!ok) {
            __syncthreads();
            continue;
        }
        bf16x8 q[R][KS];
        // waves of the same rows write the same
        const int low_most = load_rows<1, KS, R>(a, job, lane_seen, lane_depth, uniform(job.mt) * ROWS + rw * 16 * R,
                                                 s_seen + rw * 16 * R, s_low + rw * 16 * R, q);
        const int D = a.a.head_dim, len = uniform(job.e.len), total = len + uniform(job.e.count);
        const int t0 = uniform(job.t0), stages = uniform(job.t1) - t0, head = uniform(job.head);
        const int *table = a.c.tables + (size_t)uniform(job.e.seq) * a.c.max_blocks;
        const int64_t row_bytes = (int64_t)a.a.kv_heads * D * 2;
        const char *kp = a.c.pools[a.key_pool] + (int64_t)head * D * 2;
        const char *vp = a.c.pools[a.value_pool] + (int64_t)head * D * 2;
        const char *zeros = reinterpret_cast<const char *>(&past_the_head);

        auto token_of = [&](int stage, int i) {
            return (int)min((unsigned)(t0 + stage) * TK + i, (unsigned)total - 1);
        };
        // from a stage's page ids the places of its tokens, and which have none
        auto put_places = [&](int stage, int pg) {
            if (t < TK) {
                const int j = token_of(stage, t), b = divide(j, a.a.by_page);
                const bool good = in_range(pg, a.c.num_pages);
                s_off[stage & 3][t] =
                    ((int64_t)(good ? pg : 0) * a.c.page_tokens + (j - b * a.c.page_tokens)) * row_bytes;
                const uint64_t bad = __ballot(!good);
                if ((lane & 31) == 0)
                    s_lost[stage & 7][t / 32] = (uint32_t)(bad >> (lane & 32));
            }
        };
        // page ids of a stage, one load of every wave (waves past the stage's tokens repeat others')
        auto load_pages = [&](int stage) {
            const int part = w * 64 % (TK < 64 ? 64 : TK), i = (part + afresh(lane)) % TK;
            const int *p = table + divide(token_of(min(stage, stages - 1), i), a.a.by_page);
            load_to_lds4(p, lds_address(&s_page[stage & 3][part]));
        };
        auto load_rows_of = [&](int stage, auto all) {
            const uint32_t to = lds_address(mem) + stage % STAGES * 2 * HALF;
            const int l16 = afresh(lane) * 16;
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                const int at = (i * WAVES8 + w) * 1024, row = (at + l16) / ROW, slot = (at + l16) % ROW / 16;
                const int64_t off = s_off[stage & 3][row];
                const int ck = slot ^ key_order<DP>(row), cv = slot ^ value_order<DP>(row);
                const bool key = decltype(all)::value || ck * 8 < D, value = decltype(all)::value || cv * 8 < D;
                load_to_lds16<(WR < 8)>(key ? kp + off + ck * 16 : zeros, to + at);
                load_to_lds16<(WR < 8)>(vp + off + (value ? cv * 16 : 0), to + HALF + at);
            }
        };
        auto load_stage = [&](int stage) {
            if (D == DP)
                load_rows_of(stage, std::true_type());
            else
                load_rows_of(stage, std::false_type());
        };

        f32x4 o[R][NT];
        float m[R], l[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.0f;
#pragma unroll
            for (int i = 0; i < NT; ++i)
                o[r][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        for (int s = 0; s <= DEPTH && s < stages; ++s)
            if (t < TK)
                put_places(s, load_global<int>(table + divide(token_of(s, t), a.a.by_page)));
        __syncthreads();
        for (int s = 0; s < DEPTH; ++s) {
            load_pages(s + DEPTH + 1);
            if (s < stages)
                load_stage(s);
        }

        // This lane's bytes of the first block: piece `grp` of key row `col`, and 8 bytes of value row
        // 4 grp + col / 4; other pieces of the rows differ in bits of the offset, since orders are xors.
        const int key_at = col * ROW + (grp ^ key_order<DP>(col)) * 16;
        const int value_row = grp * 4 + (col >> 2);
        const int value_at = value_row * ROW + ((col >> 1 & 1) ^ value_order<DP>(value_row)) * 16 + (col & 1) * 8;

        // Stage i and the page ids loaded with it are there (what came after may be under way), and all
        // waves have read what they need of stage i - 1.
        auto begin_stage = [&](int i) {
            if (i + DEPTH <= stages)
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((DEPTH - 1) * (2 * LOADS + 1))
                             : "memory");
            else
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            load_pages(i + PAGE_AHEAD);
            if (i + DEPTH < stages)
                load_stage(i + DEPTH);
            if (i + DEPTH + 1 < stages && t < TK)
                put_places(i + DEPTH + 1, s_page[i + DEPTH + 1 & 3][t]);
        };
        u32x4 kf[KS][2];
        int lost_here;
        auto read_keys = [&](int i, int kb) {
            const int b0 = (kg * KB + kb) * 32, at = key_at + i % STAGES * 2 * HALF + b0 * ROW;
            lost_here = (int)s_lost[i & 7][b0 / 32];
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    kf[k][x] = *reinterpret_cast<const u32x4 *>(mem + (at ^ k * 64) + x * 16 * ROW);
        };
        f32x4 sc[R][2];
        s16x4 vf[EARLY][2];
        auto read_value = [&](int block_at, int x, int h) {
            const char *at = mem + ((value_at + block_at) ^ x * 32) + HALF + h * 16 * ROW;
            return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4 *)at);
        };
        // scores of the block whose keys are in kf, and in the plain loop the first of its values
        auto read_early = [&](int block_at) {
#pragma unroll
            for (int x = 0; x < EARLY; ++x)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    vf[x][h] = read_value(block_at, x, h);
        };
        auto score = [&] {
            __builtin_amdgcn_s_setprio(1);
#pragma unroll
            for (int r = 0; r < R; ++r)
                sc[r][0] = sc[r][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < KS; ++k)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int r = 0; r < R; ++r)
                        sc[r][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kf[k][x]), q[r][k],
                                                                           sc[r][x], 0, 0, 0);
            __builtin_amdgcn_s_setprio(0);
        };
        // the weights' product with the values; out of the plain loop rows that `odd` names count as 0
        auto add_values = [&](auto plain, int block_at, uint32_t odd) {
            constexpr bool PLAIN = decltype(plain)::value;
            __builtin_amdgcn_s_setprio(1);
            bf16x8 p[R];
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int y = 0; y < 8; ++y)
                    p[r][y] = (__bf16)sc[r][y / 4][y & 3];
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                s16x4 v[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    v[h] = PLAIN && x < EARLY ? vf[x < EARLY ? x : 0][h] : read_value(block_at, x, h);
                    if constexpr (!PLAIN)
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            v[h][y] = odd >> (h * 16 + grp * 4 + y) & 1 ? (short)0 : v[h][y];
                }
                const bf16x8 vt =
                    __builtin_bit_cast(bf16x8, __builtin_shufflevector(v[0], v[1], 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
                for (int r = 0; r < R; ++r)
                    o[r][x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vt, p[r], o[r][x], 0, 0, 0);
                // one after another: all at once would take more registers than there are
                if constexpr (!PLAIN)
                    __builtin_amdgcn_sched_barrier(0);
            }
        };
        // A block that some row does not see all of, or whose maximum the running one must follow, or whose is FAR.
        auto slow_block = [&](int block_at, int j0, uint32_t lost) {
            score();
            uint32_t odd = 0;
            // as in k_attend: rows of values with an infinity or a NaN are added one by one
            if ((unsigned)j0 + 32 > (unsigned)len || lost != 0 || j0 < low_most) {
#pragma unroll 1
                for (int x = 0; x < 32 * PIECES / 64; ++x) {
                    const int p = x * 64 + lane, row = p / PIECES;
                    const u32x4 v = *reinterpret_cast<const u32x4 *>(mem + block_at + HALF + p * 16);
                    const bool mine = odd_word<1>(v[0]) || odd_word<1>(v[1]) || odd_word<1>(v[2]) || odd_word<1>(v[3]);
                    for (uint64_t all = __ballot(mine); all != 0; all &= all - 1)
                        odd |= 1u << uniform(__shfl(row, __builtin_ctzll(all)));
                }
            }
            uint32_t vis[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int row = rw * 16 * R + r * 16 + col;
                vis[r] = visible(len, s_low[row], s_seen[row], j0, lost);
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        sc[r][x][y] = vis[r] >> (grp * 4) & (1u << (x * 16 + y)) ? sc[r][x][y] : -INFINITY;
            }
            follow<2, NT, R>(sc, o, m, l, a.c1);
            if (any_far<R>(m, a.far))
                weigh<true, 2, R>(sc, m, l, a.c1, a.far, LAG);
            else
                weigh<false, 2, R>(sc, m, l, a.c1, a.far, LAG);
#pragma unroll 1
            for (uint32_t left = odd; left != 0; left &= left - 1) {
                const int key = __builtin_ctz(left);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    float pr = 0.0f;
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            pr = key / 16 == x && (key & 3) == y ? sc[r][x][y] : pr;
                    pr = __shfl(pr, (key >> 2 & 3) * 16 + col);
                    const bool sees = vis[r] >> key & 1;
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        const u32x2 four = *reinterpret_cast<const u32x2 *>(
                            mem + block_at + HALF + key * ROW + ((x * 2 + grp / 2) ^ value_order<DP>(key)) * 16 +
                            (grp & 1) * 8);
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            const float v = __uint_as_float(y & 1 ? four[y / 2] & 0xffff0000u : four[y / 2] << 16);
                            o[r][x][y] = sees ? o[r][x][y] + pr * v : o[r][x][y];
                        }
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
            add_values(std::false_type(), block_at, odd);
        };

        // The loop over blocks leaves those that need more than the plain steps to slow_block, so that
        // its registers are changed in place.
        const float slack = LAG / a.c1;
        const int blocks = stages * KB;
        const bool late = w >= WAVES8 / 2;
        int begun = -1;
        for (int b = 0; b < blocks; ++b) {
            int block_at = 0, j0 = 0;
            // every way out is before the sums change
            for (;; ++b) {
                const int i = b / KB, kb = b - i * KB;
                if (b < blocks && begun != i) {
                    begun = i;
                    begin_stage(i);
                }
                const int b0 = (kg * KB + kb) * 32;
                j0 = (int)((unsigned)(t0 + i) * TK + b0);
                block_at = i % STAGES * 2 * HALF + b0 * ROW;
                if (b >= blocks || (unsigned)j0 + 32 > (unsigned)len || j0 < low_most)
                    break;
                read_keys(i, kb);
                if constexpr (!SHIFT)
                    read_early(block_at);
                score();
                bool grew = uniform(lost_here) != 0;
#pragma unroll
                for (int r = 0; r < R; ++r)
                    grew |= tile_max<2>(sc[r]) > (fabsf(m[r]) < a.far ? m[r] + slack : -INFINITY);
                if (__ballot(grew) != 0)
                    break;
                if (SHIFT && late && kb == KB - 1 && i + 1 < stages) {
                    begun = i + 1;
                    begin_stage(i + 1);
                }
                if constexpr (SHIFT)
                    read_early(block_at);
                weigh<false, 2, R>(sc, m, l, a.c1, a.far, LAG);
                add_values(std::true_type(), block_at, 0);
            }
            if (b < blocks && (unsigned)j0 < (unsigned)total) {
                read_keys(b / KB, b % KB);
                slow_block(block_at, j0, (uint32_t)uniform(lost_here));
            }
        }
        // nothing is under way to LDS, and all have read it
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        float(*s_o)[PITCH] = reinterpret_cast<float(*)[PITCH]>(mem);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float sum = row_sum(l[r]);
            const int at = w * 16 * R + r * 16 + col;
            if (grp == 0)
                s_ml[at] = make_float2(m[r] == -INFINITY ? -INFINITY
                                                         : __builtin_fmaf(m[r], a.c1 * QUARTER, LAG * QUARTER), sum);
#pragma unroll
            for (int x = 0; x < NT; ++x)
                *reinterpret_cast<f32x4 *>(&s_o[at][x * 16 + grp * 4]) = o[r][x];
        }
        __syncthreads();
        // waves rw, rw + WR, ... hold the same rows
        finish<1, ATTN_WIDE_WG, PITCH>(a, job, ROWS, s_o, s_ml, KG, ROWS);
        __syncthreads();
    }
}

// LG lanes join what the parts of one row left, 4 elements each; eight parts' loads under way at once.
// SPLIT: a workgroup has one row, and its groups of lanes every GROUPS-th part, joined in their order.
// Rows of one part are done.  Bound by memory where many rows are split (65536 rows of 128 in two
// parts: 29 us for 84 MB), by the launch and the latency of its loads else (32 rows of 8 parts: 4 us).
//
// Up to JOIN_SPLIT rows to a compute unit are split: attend of 5 nodes over 250001 tokens (160 rows of 32
// parts) 182 -> 178 us, of one node 199 -> 190 us; for 2048 rows of two parts it is 213 us against 211.
constexpr int JOIN_SPLIT = 4;

template <int DT, int LG, bool SPLIT>
__global__ __launch_bounds__(ATTN_WG) void k_attend_join(AttnArgs a, int rows_per_tile)
{
    constexpr int ES = Tile<DT>::ES, GROUPS = ATTN_WG / LG, STEP = SPLIT ? GROUPS : 1;
    __shared__ f32x4 s_acc[SPLIT ? GROUPS : 1][LG];
    __shared__ float2 s_ml[SPLIT ? GROUPS : 1];
    const int lane = threadIdx.x & (LG - 1), group = threadIdx.x / LG;
    const uint32_t per = (uint32_t)a.nv.max_count * a.a.q_heads;       // the launch's work-items fit 32 bits
    const uint32_t at = SPLIT ? blockIdx.x : blockIdx.x * GROUPS + group;
    const int i = (int)(at / per), rest = (int)(at - i * per);
    if (i >= a.nv.n)
        return;
    const AttnPlan p = a.a.plan[i];
    const int sound = a.a.sound[i];
    const double share = *a.a.share;
    const int node = rest / a.a.q_heads, qh = rest - node * a.a.q_heads;
    if (node >= p.count)
        return;
    const int D = a.a.head_dim, head = divide(qh, a.a.by_group);
    const int gr = node * a.a.group + qh - head * a.a.group, mt = gr / rows_per_tile, row = gr - mt * rows_per_tile;
    const double base = p.base + (double)(head * p.tiles_of_rows + mt) * p.counted + (p.counted - p.tiles);
    const int w0 = (int)(base / share), parts = (int)((base + (p.tiles - 1)) / share) - w0 + 1;
    if (parts < 2 || !sound)
        return;
    const int d = lane * 4 < D ? lane * 4 : 0;
    float top = -INFINITY, z = 0.0f;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int c0 = SPLIT ? group : 0; c0 < parts; c0 += 8 * STEP) {
        float2 ml[8];
        f32x4 v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            // the last part again where there is none, without weight
            const int part = min(c0 + c * STEP, parts - 1);
            const int64_t kept = (int64_t)(2 * (w0 + part) + (part == 0)) * rows_per_tile + row;
            ml[c] = a.a.part_ml[kept];
            v[c] = load_global<f32x4>(a.a.part_o + kept * D + d);
        }
        const float was = top;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            top = fmaxf(top, ml[c].x);
        const float old = scale_down(was, top);
        z *= old;
        acc *= old;
#pragma unroll
        for (int c = 0; c < 8; ++c)
            if (c0 + c * STEP < parts) {
                const float f = scale_down(ml[c].x, top);
                z += f * ml[c].y;
                acc += f * v[c];
            }
    }
    if constexpr (SPLIT) {
        s_acc[group][lane] = acc;
        if (lane == 0)
            s_ml[group] = make_float2(top, z);
        __syncthreads();
        if (group > 0)
            return;
        for (int g = 1; g < min(parts, GROUPS); ++g)
            top = fmaxf(top, s_ml[g].x);
        z = 0.0f;
        acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int g = 0; g < min(parts, GROUPS); ++g) {
            const float2 ml = s_ml[g];
            const float f = scale_down(ml.x, top);
            z += f * ml.y;
            acc += f * s_acc[g][lane];
        }
    }
    if (lane * 4 >= D)
        return;
    char *to = a.out + (int64_t)(p.start + node) * a.out_stride + ((int64_t)qh * D + lane * 4) * ES;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const float o = z == 0.0f ? 0.0f : acc[x] / z;
        if constexpr (DT == 1)
            reinterpret_cast<__bf16 *>(to)[x] = (__bf16)o;
        else
            reinterpret_cast<float *>(to)[x] = o;
    }
    if (a.lse && lane == 0)
        a.lse[(int64_t)(p.start + node) * a.a.q_heads + qh] = log_sum(top, z);
}

template <int LG> void join_with(hipStream_t st, bool bf16, const AttnArgs &a, int rows, int64_t joined)
{
    const bool split = joined <= JOIN_SPLIT * a.a.num_cus;
    const unsigned groups = (unsigned)(split ? joined : (joined * LG + ATTN_WG - 1) / ATTN_WG);
    auto join = split ? (bf16 ? k_attend_join<1, LG, true> : k_attend_join<0, LG, true>)
                      : (bf16 ? k_attend_join<1, LG, false> : k_attend_join<0, LG, false>);
    join<<<groups, ATTN_WG, 0, st>>>(a, rows);
}

// The launch of a form for tiles of `rows` rows.
template <typename K> hipError_t attend_with(hipStream_t st, K kernel, AttnArgs a, int threads, int rows, int per_cu)
{
    a.units = (std::min(a.a.num_cus * per_cu, ATTN_MAX_UNITS) + 7) / 8 * 8;
    kernel<<<a.units, threads, 0, st>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    const int64_t joined = (int64_t)a.nv.n * a.nv.max_count * a.a.q_heads;
    if (joined == 0)
        return hipSuccess;
    const bool bf16 = a.a.dtype == 1;
    if (a.a.head_dim <= 64)
        join_with<16>(st, bf16, a, rows, joined);
    else if (a.a.head_dim <= 128)
        join_with<32>(st, bf16, a, rows, joined);
    else
        join_with<64>(st, bf16, a, rows, joined);
    return hipGetLastError();
}

}  // namespace

// Two tiles of rows to each workgroup of a launch: 32 rows of k_attend, 256 of k_attend_wide.
int64_t attend_kept_rows(int num_cus)
{
    return 2 * std::max<int64_t>(ATTN_MAX_UNITS * 32, (num_cus + 7) / 8 * 8 * 256);
}

hipError_t launch_attend(hipStream_t st, const CacheView &c, const AttnShape &s, const NodesView &nodes,
                         int key_pool, int value_pool, float scale, int window, const void *q,
                         int64_t q_stride, void *out, int64_t out_stride, float *lse, int *status)
{
    const int D = s.head_dim, M = nodes.max_count * s.group, es = s.dtype == 1 ? 2 : 4;
    const float c1 = scale == 0.0f ? 1.0f : fabsf(scale) * LOG2E;
    AttnArgs a = {c, s, nodes, key_pool, value_pool, c1, FAR / c1,
                  scale > 0.0f ? 1.0f : scale < 0.0f ? -1.0f : 0.0f, window, static_cast<const char *>(q),
                  q_stride * es, static_cast<char *>(out), out_stride * es, lse, status, 0};
    // Forms with tiles of as many rows as there are, or the largest.  Up to 16 rows k_attend begins and ends
    // faster, k_attend_wide reads long sequences faster, and the lengths are not known here: in us, k_attend
    // and k_attend_wide, heads of 128 and 4 rows, one sequence of 1000 tokens 13.3 and 15.6, of 250001 190 and 176;
    // 64 sequences of 50 to 400 tokens 30 and 37, of 300 to 2000 72 and 72, of 300 to 8200 211 and 197; the
    // last with heads of 64 224 and 194, of 80 198 and 203, of 256 203 and 224.
    // k_attend has as many workgroups on a compute unit as its registers allow (float32 heads of 64, when it
    // was chosen: 3, 70 us; 2, 79 us; 4, 100 us for spills).  Float32 has no other form: 16 sequences of 1000 to 5000
    // tokens, 4 key heads of 128, 32, 64, 128 and 512 rows: 78, 115, 187 and 598 us, where its matrix
    // instructions alone take 19, 38, 75 and 300 and the bytes 40; every 32 rows (16 of heads of 256) read them again.
    // k_attend_wide has what its registers and 160 KB of LDS allow, and of that the fastest, in us for 64
    // sequences of 300 to 8200 tokens (waves over the rows x rows of a wave, tokens x number of stages):
    //   heads of 64:  32 rows  2 x 16, 128 x 4: 206;  x 2: 229
    //                 64 rows  2 x 32, 128 x 4: 236;  4 x 16, 64 x 4: 248
    //                128 rows  4 x 32, 128 x 4: 318;  64 x 4: 342;  8 x 16, 64 x 4: 407
    //                256 rows  8 x 32, 128 x 4: 271;  64 x 4: 288  (half the heads)
    //   of 128:       64 rows  4 x 16,  64 x 4: 226;  2 x 32, 128 x 2: 250
    //                128 rows  4 x 32,  64 x 4: 270;  8 x 16, 64 x 4: 298;  32 x 4: 307
    //                256 rows  8 x 32,  64 x 4: 501;  32 x 4: 527  (16 sequences of 512 rows)
    //   of 256:      128 rows  8 x 16,  32 x 4: 280;  64 x 2: 305
#define NARROW(DT, DP, VW, R, OCC) attend_with(st, k_attend<DT, DP, VW, R, OCC>, a, ATTN_WG, 16 * R, OCC < 2 ? 2 : OCC)
#define WIDE(DP, R, WR, KB, STAGES) \
    attend_with(st, k_attend_wide<DP, R, WR, KB, STAGES>, a, ATTN_WIDE_WG, 16 * R * WR, 1)
    if (s.dtype == 0) {
        if (D <= 64)
            return M <= 16 ? NARROW(0, 64, 4, 1, 3) : NARROW(0, 64, 4, 2, 2);
        if (D <= 128)
            return M <= 16 ? NARROW(0, 128, 4, 1, 2) : NARROW(0, 128, 4, 2, 1);
        return NARROW(0, 256, 4, 1, 1);
    }
    if (M <= 16)
        return D <= 64 ? NARROW(1, 64, 4, 1, 3) : D <= 128 ? NARROW(1, 128, 8, 1, 2) : NARROW(1, 256, 8, 1, 1);
    if (D <= 64)
        return M <= 32 ? WIDE(64, 1, 2, 1, 4) : M <= 64 ? WIDE(64, 2, 2, 1, 4)
             : M <= 128 ? WIDE(64, 2, 4, 2, 4) : WIDE(64, 2, 8, 4, 4);
    if (D <= 128)
        return M <= 32 ? WIDE(128, 1, 2, 1, 2) : M <= 64 ? WIDE(128, 1, 4, 1, 4)
             : M <= 128 ? WIDE(128, 2, 4, 1, 4) : WIDE(128, 2, 8, 2, 4);
    return M <= 64 ? WIDE(256, 1, 4, 1, 2) : WIDE(256, 1, 8, 1, 4);
#undef NARROW
#undef WIDE
}

// ------------------------------------------------------------------ append

namespace {

// cos and sin of position * inv_freq: the angle in turns in fp64, what is left of whole turns in fp32.
__device__ inline float2 turn(int position, float inv_freq)
{
    const double x = (double)position * (double)inv_freq * 0.15915494309189533577;
    const float h = 2.0f * (float)(x - rint(x));
    float s, c;
    sincospif(h, &s, &c);
    return make_float2(c, s);
}

constexpr int APPEND_TOKENS = 4;                   // of an entry to a workgroup
constexpr int APPEND_PAIRS = ATTN_MAX_HEAD_DIM / 2;

struct AppendArgs {
    CacheView c;
    AttnShape a;
    NodesView nv;
    RotationView rot;
    int key_pool, value_pool;
    const char *k, *v, *q;
    char *rotated;
    int64_t k_stride, v_stride, q_stride, rotated_stride;   // bytes
    int *status;
    int tokens;          // of an entry to a group of workgroups
    int split;           // workgroups of a group
    FastDiv by_group;    // groups of an entry, times split
    FastDiv by_token;    // pieces of a token
    FastDiv by_head;     // pieces of a rotated head
};

template <int DT, int N> __device__ inline void load_piece(const char *p, float (&x)[N])
{
    if constexpr (N == Elt<DT>::EPV) {
        const u32x4 v = load_global<u32x4_any>(p);
        Elt<DT>::unpack(make_uint4(v[0], v[1], v[2], v[3]), x);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if constexpr (DT == 1)
                x[i] = __uint_as_float((uint32_t)load_global<uint16_t>(p + 2 * i) << 16);
            else
                x[i] = load_global<float>(p + 4 * i);
    }
}

template <int DT, int N> __device__ inline void store_piece(char *p, const float (&x)[N])
{
    if constexpr (DT == 0 && N == 4) {
        store_global<u32x4_any>(p, u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                                         __float_as_uint(x[3])});
    } else if constexpr (DT == 1 && N == 8) {
        bf16x8 v;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = (__bf16)x[i];
        store_global<u32x4_any>(p, __builtin_bit_cast(u32x4, v));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if constexpr (DT == 1)
                store_global<__bf16>(p + 2 * i, (__bf16)x[i]);
            else
                store_global<float>(p + 4 * i, x[i]);
    }
}

template <int DT, bool VEC> __device__ inline void copy_piece(char *to, const char *from)
{
    if constexpr (VEC)
        store_global<u32x4_any>(to, load_global<u32x4_any>(from));
    else if constexpr (DT == 1)
        store_global<uint16_t>(to, load_global<uint16_t>(from));
    else
        store_global<uint32_t>(to, load_global<uint32_t>(from));
}

// Pair (x, y) number p of a head, at position n, turns by the angle n inv_freq[p]:
// (x cos - y sin, y cos + x sin).  A rotated piece holds 16 bytes of both halves of a head (of
// neighbouring pairs: 16 bytes), the others 16 bytes, at any address of the element's alignment;
// without VEC, where the rotated part is no whole number of them, one pair and one element.  A token's
// pieces: its query heads', its key heads', its values'.  Angles of a token are computed once, into LDS.
//
// Bound by memory, a few tokens by the call: 13800 tokens of 32 query and 8 key heads of 128 in
// bfloat16: 76.5 us, 4.4 TB/s read and written (a large copy 5.0); 2112 tokens in 256 entries 12.7 us; one
// 8.3 us.  Four tokens to a workgroup: with 2 it is 78.7 us, with 8 83.8, with 16 101.  Without VEC it is bound by
// its loads of one element: heads of 80, 13800 tokens, 80 rotated dimensions 50.5 us, 40 and 20 130 and 142.
template <int DT, bool VEC, bool INTER>
__global__ __launch_bounds__(ATTN_WG) void k_append(AppendArgs a)
{
    constexpr int ES = Elt<DT>::BYTES, N = VEC ? Elt<DT>::EPV : 1;
    constexpr int PAIRS = INTER && VEC ? N / 2 : N;      // pairs of a rotated piece
    __shared__ float2 cs[APPEND_TOKENS][APPEND_PAIRS];
    __shared__ int64_t place[APPEND_TOKENS];
    __shared__ int depth_of[MAX_NODES];
    const int group = divide((int)blockIdx.x, a.by_group);
    const int within = (int)blockIdx.x - group * (int)a.by_group.d;
    const int first = within / a.split * a.tokens, part = within - within / a.split * a.split;
    const int t = threadIdx.x, i = group;

    const Entry e = load_entry(a.c, a.nv, i);
    bool ok = e.count >= 0;
    if (ok && a.nv.parents) {
        uint64_t seen;
        int depth;
        ok = lane_node(a.nv.parents + e.start, e.count, 0, seen, depth);
        if (ok && t < MAX_NODES)
            depth_of[t] = depth;
    }
    if (ok && a.nv.seqs) {
        bool named = false;
        for (int j = t; j < i; j += ATTN_WG)
            named |= a.nv.seqs[j] == e.seq;
        ok = !__syncthreads_or(named);
    }
    if (a.status && within == 0 && t == 0)
        a.status[i] = ok ? 0 : -1;
    if (!ok || first >= e.count)
        return;
    __syncthreads();
    const int tokens = min(a.tokens, e.count - first), dims = a.rot.dims, half = dims / 2;
    const int D = a.a.head_dim, Hk = a.a.kv_heads, Hq = a.q ? a.a.q_heads : 0;
    const int64_t row_bytes = (int64_t)Hk * D * ES;
    if (t < tokens) {
        const int j = e.len + first + t, b = divide(j, a.a.by_page);
        const int pg = a.c.tables[(size_t)e.seq * a.c.max_blocks + b];
        place[t] = in_range(pg, a.c.num_pages)
                       ? ((int64_t)pg * a.c.page_tokens + (j - b * a.c.page_tokens)) * row_bytes
                       : -1;
    }
    for (int x = t; x < tokens * half; x += ATTN_WG) {
        const int tk = x / half, p = x - tk * half;
        const int depth = a.nv.parents ? depth_of[first + tk] : first + tk;
        cs[tk][p] = turn(e.len + depth, a.rot.inv_freq[p]);
    }
    __syncthreads();

    char *kp = a.c.pools[a.key_pool], *vp = a.c.pools[a.value_pool];
    const int per_token = (int)a.by_token.d, per_head = (int)a.by_head.d, turned = half / PAIRS;
    for (int x = part * ATTN_WG + t; x < tokens * per_token; x += a.split * ATTN_WG) {
        const int tk = divide(x, a.by_token), y = x - tk * per_token;
        const int64_t row = e.start + first + tk;
        const int64_t at = place[tk];
        if (y >= (Hq + Hk) * per_head) {
            const int64_t o = (int64_t)(y - (Hq + Hk) * per_head) * N * ES;
            if (at >= 0)
                copy_piece<DT, VEC>(vp + at + o, a.v + row * a.v_stride + o);
            continue;
        }
        int h = divide(y, a.by_head);
        const int u = y - h * per_head;
        const char *from;
        char *to;
        if (h < Hq) {
            from = a.q + row * a.q_stride;
            to = a.rotated + row * a.rotated_stride;
        } else {
            h -= Hq;
            if (at < 0)
                continue;
            from = a.k + row * a.k_stride;
            to = kp + at;
        }
        from += (int64_t)h * D * ES;
        to += (int64_t)h * D * ES;
        if (u >= turned) {
            const int64_t o = (int64_t)(dims + (u - turned) * N) * ES;
            copy_piece<DT, VEC>(to + o, from + o);
        } else if constexpr (INTER) {
            float v[2 * PAIRS];
            const int64_t o = (int64_t)u * 2 * PAIRS * ES;
            load_piece<DT>(from + o, v);
#pragma unroll
            for (int p = 0; p < PAIRS; ++p) {
                const float2 f = cs[tk][u * PAIRS + p];
                const float g = v[2 * p], b = v[2 * p + 1];
                v[2 * p] = __builtin_fmaf(g, f.x, -(b * f.y));
                v[2 * p + 1] = __builtin_fmaf(b, f.x, g * f.y);
            }
            store_piece<DT>(to + o, v);
        } else {
            float v[N], z[N];
            const int64_t o = (int64_t)u * N * ES, far = (int64_t)half * ES;
            load_piece<DT>(from + o, v);
            load_piece<DT>(from + o + far, z);
#pragma unroll
            for (int p = 0; p < N; ++p) {
                const float2 f = cs[tk][u * N + p];
                const float g = v[p], b = z[p];
                v[p] = __builtin_fmaf(g, f.x, -(b * f.y));
                z[p] = __builtin_fmaf(b, f.x, g * f.y);
            }
            store_piece<DT>(to + o, v);
            store_piece<DT>(to + o + far, z);
        }
    }
}

template <int DT> hipError_t append_with(hipStream_t st, AppendArgs &a, bool vec)
{
    const int n_el = vec ? Elt<DT>::EPV : 1, D = a.a.head_dim, dims = a.rot.dims, Hk = a.a.kv_heads;
    const int turned = dims / 2 / (a.rot.interleaved && vec ? n_el / 2 : n_el);
    const int per_head = turned + (D - dims) / n_el;
    const int per_token = ((a.q ? a.a.q_heads : 0) + Hk) * per_head + Hk * D / n_el;
    a.by_head = fast_div(per_head);
    a.by_token = fast_div(per_token);
    a.tokens = std::max(std::min(APPEND_TOKENS, a.nv.max_count), 1);
    const int64_t groups = std::max<int64_t>(((int64_t)a.nv.max_count + a.tokens - 1) / a.tokens, 1);
    // a piece to a thread where there are few tokens
    const int64_t want = 2 * (int64_t)a.a.num_cus / std::max<int64_t>(1, groups * a.nv.n);
    const int64_t most = ((int64_t)a.tokens * per_token + ATTN_WG - 1) / ATTN_WG;
    a.split = (int)std::max<int64_t>(1, std::min(want, most));
    const int64_t per_entry = groups * a.split;
    if (per_entry * a.nv.n * ATTN_WG > 0xffffffffll)
        return hipErrorInvalidConfiguration;
    a.by_group = fast_div((int)per_entry);
    const unsigned grid = (unsigned)(per_entry * a.nv.n);
    if (vec)
        a.rot.interleaved ? k_append<DT, true, true><<<grid, ATTN_WG, 0, st>>>(a)
                          : k_append<DT, true, false><<<grid, ATTN_WG, 0, st>>>(a);
    else
        a.rot.interleaved ? k_append<DT, false, true><<<grid, ATTN_WG, 0, st>>>(a)
                          : k_append<DT, false, false><<<grid, ATTN_WG, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_append(hipStream_t st, const CacheView &c, const AttnShape &s, const NodesView &nodes,
                         const RotationView &rot, int key_pool, int value_pool, const void *k,
                         int64_t k_stride, const void *v, int64_t v_stride, const void *q,
                         int64_t q_stride, void *rotated, int64_t rotated_stride, int *status)
{
    const int es = s.dtype == 1 ? 2 : 4, epv = 16 / es;
    AppendArgs a = {c, s, nodes, rot, key_pool, value_pool, static_cast<const char *>(k),
                    static_cast<const char *>(v), static_cast<const char *>(q),
                    static_cast<char *>(rotated), k_stride * es, v_stride * es, q_stride * es,
                    rotated_stride * es, status, 0, 0, {}, {}, {}};
    const bool vec = (rot.interleaved ? rot.dims : rot.dims / 2) % epv == 0;
    return s.dtype == 1 ? append_with<1>(st, a, vec) : append_with<0>(st, a, vec);
}

}  // namespace sv
