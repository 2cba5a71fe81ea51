// Draws and verification from laws cut by top-k, top-p and min-p (gfx950).
//
// The law of a row x with temperature T, top-k k, top-p p and min-p m: order the ids by x
// descending, ties lowest id first; w_i = exp((x_i - max x) / T); S_k = the first k ids; S_p =
// the ids of S_k whose exclusive prefix sum of w, in that order, is below p * sum(S_k) (the first
// always); S = the ids of S_p with w_i >= m; P(i) = w_i / Z on S, Z = sum(S).
//
// Every step keeps a prefix of the order, so S itself is a prefix: it is the ids above a cut
// value plus the lowest ids among those equal to it.  A row is therefore described by (cut value,
// last id kept at that value, Z), RowCut, and no row is ever sorted.
//
//   k_filter_sample   one 1024-thread workgroup per row: its RowCut, then the inverse-CDF draw
//   k_filter_rows     the RowCut of every target and draft row of a verify
//   k_filter_verify   one workgroup per sequence: accept tests, first rejection, residual draw
//
// The cut has to be the exact one, because ids are compared for equality with the definition: all
// weights and sums are fp64.
#include <float.h>

#include "sv_device.h"
#include "sv_internal.h"

namespace sv {

namespace {

constexpr int FWG = FILTER_WG;
constexpr int FWAVES = FWG / 64;

// Order-preserving 32-bit key of a logit: larger value, larger key; -0 and +0 are one key.
__device__ inline uint32_t order_key(float x)
{
    const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ inline float key_value(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

constexpr uint32_t KEY_POS_INF = 0xff800000u;   // order_key(+inf); NaNs lie above it
constexpr uint32_t KEY_NEG_INF = 0x007fffffu;   // order_key(-inf); negative NaNs lie below it

__device__ inline double weight(float x, float m, double c) { return exp2(((double)x - (double)m) * c); }

struct Params {
    double c;       // log2(e) / T
    double p, m;
    int k;          // 1..V
    bool ok;
};

// One row's or sequence's parameters: absent arrays cut nothing.  T = 0 is the first id of the
// order, which is k = 1 at any temperature.
__device__ inline Params load_params(const FilterPtrs &f, int i, int V)
{
    Params q;
    const float T = f.temperature ? f.temperature[i] : 1.0f;
    const int k = f.top_k ? f.top_k[i] : 0;
    const float p = f.top_p ? f.top_p[i] : 1.0f;
    const float m = f.min_p ? f.min_p[i] : 0.0f;
    q.ok = T >= 0.0f && T <= FLT_MAX && p >= 0.0f && p <= 1.0f && m >= 0.0f && m <= 1.0f;
    q.c = T == 0.0f ? 1.4426950408889634074 : 1.4426950408889634074 / (double)T;
    q.k = T == 0.0f ? 1 : (k <= 0 || k > V) ? V : k;
    q.p = (double)p;
    q.m = (double)m;
    return q;
}

// Sum over the workgroup, the same bits in every thread (fixed order).
template <typename T> __device__ T block_sum(T v, T *lds)
{
    v = wave_sum_lds(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    T s = lds[0];
    for (int i = 1; i < FWAVES; ++i)
        s += lds[i];
    return s;
}

__device__ inline uint32_t block_max(uint32_t v, uint32_t *lds)
{
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        v = max(v, (uint32_t)__shfl_xor((int)v, o));
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        lds[threadIdx.x >> 6] = v;
    __syncthreads();
    uint32_t s = lds[0];
    for (int i = 1; i < FWAVES; ++i)
        s = max(s, lds[i]);
    return s;
}

struct RedLds {
    double d[FWAVES];
    uint32_t u[FWAVES];
    int i[FWAVES];
};

__device__ inline bool kept(uint32_t key, int id, const RowCut &r)
{
    return key > r.cut || (key == r.cut && id <= r.tie);
}

// The row's cut by bisection on the order keys: every step is one pass over the row that counts
// or sums what lies above a key.  Exact for any row; 32 passes per active cut.
template <int DT>
__device__ RowCut cut_by_bisection(const char *row, int V, const Params &q, RedLds &lds)
{
    RowCut r;
    const int t = threadIdx.x;
    uint32_t mx = 0;
    int bad = 0;
    for (int i = t; i < V; i += FWG) {
        const uint32_t k = order_key(Elt<DT>::one(row, i));
        bad |= (k >= KEY_POS_INF) | (k < KEY_NEG_INF);
        mx = max(mx, k);
    }
    mx = block_max(mx, lds.u);
    bad = block_sum(bad, lds.i);
    r.state = q.ok && !bad && mx > KEY_NEG_INF ? CUT_READY : CUT_NONE;
    r.max = key_value(mx);
    r.c = q.c;
    r.cut = KEY_NEG_INF;                            // no key lies below it: all ids
    r.tie = V;
    r.z = 0.0;
    if (r.state == CUT_NONE)
        return r;
    const float M = r.max;
    auto count_ge = [&](uint32_t key) {
        int n = 0;
        for (int i = t; i < V; i += FWG)
            n += order_key(Elt<DT>::one(row, i)) >= key;
        return block_sum(n, lds.i);
    };
    // the last kept id among those equal to the cut, the n-th of them
    auto nth_tie = [&](uint32_t key, int n) {
        int lo = 0, hi = V - 1;
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            int c = 0;
            for (int i = t; i <= mid; i += FWG)
                c += order_key(Elt<DT>::one(row, i)) == key;
            if (block_sum(c, lds.i) >= n)
                hi = mid;
            else
                lo = mid + 1;
        }
        return lo;
    };
    // sum of the weights kept by r with keys above `key`
    auto mass_above = [&](uint32_t key) {
        double s = 0.0;
        for (int i = t; i < V; i += FWG) {
            const float x = Elt<DT>::one(row, i);
            const uint32_t k = order_key(x);
            if (k > key && kept(k, i, r))
                s += weight(x, M, r.c);
        }
        return block_sum(s, lds.d);
    };
    if (q.k < V) {
        uint32_t lo = 0, hi = mx;                   // count_ge(lo) >= k
        while (lo < hi) {
            const uint32_t mid = hi - ((hi - lo) >> 1);
            if (count_ge(mid) >= q.k)
                lo = mid;
            else
                hi = mid - 1;
        }
        r.cut = lo;
        r.tie = nth_tie(lo, q.k - count_ge(lo + 1));
    }
    r.z = mass_above(0);
    if (q.p < 1.0) {
        const double goal = q.p * r.z;
        uint32_t lo = r.cut, hi = mx;               // the smallest key with mass above it < goal
        while (lo < hi) {
            const uint32_t mid = lo + ((hi - lo) >> 1);
            if (mass_above(mid) < goal)
                hi = mid;
            else
                lo = mid + 1;
        }
        const double over = mass_above(lo);
        const double n = ceil((goal - over) / weight(key_value(lo), M, r.c));
        const int tie = nth_tie(lo, n < 1.0 ? 1 : n > (double)V ? V : (int)n);
        r.tie = lo == r.cut ? min(tie, r.tie) : tie;
        r.cut = lo;
        r.z = mass_above(0);
    }
    if (weight(key_value(r.cut), M, r.c) < q.m) {
        uint32_t lo = r.cut, hi = mx;               // the smallest key of weight >= m
        while (lo < hi) {
            const uint32_t mid = lo + ((hi - lo) >> 1);
            if (weight(key_value(mid), M, r.c) >= q.m)
                hi = mid;
            else
                lo = mid + 1;
        }
        r.cut = lo;
        r.tie = V;
        r.z = mass_above(0);
    }
    return r;
}

// ------------------------------------------------------------------ bfloat16: the cut by counting
//
// A bfloat16 row has few distinct values, so its cut comes from how often each occurs: one pass
// counts the bit patterns in LDS, and every sum above is a sum over patterns of count * weight.
// The counts are integers, so the cut is exact and the same in every run, and the exponentials
// are one per pattern instead of one per logit.
//
// Counted are the patterns with 2^-24 <= |x| < 2^8: 4096 magnitudes and two signs, 32 KiB.  What
// lies outside is rare in logits and kept apart: zeros (a count), up to 63 other values (a list),
// and values <= -2^8, of which only the largest is noted: beside a row's maximum they weigh
// nothing unless all of the row is low.  A row that this does not cover goes to cut_by_bisection.

constexpr uint32_t HLO = 103u << 7;        // pattern of 2^-24
constexpr int HMAG = 4096;
constexpr int HBINS = 2 * HMAG;            // bin = 2 * (magnitude - HLO) + sign
constexpr int HX = 64;                     // values outside the window kept apart
// Bins are put in order 64 at a time: tile 0 the values above the window, 1..64 the positive
// bins, 65 the values around zero, 66..129 the negative bins.
constexpr int NTILES = 2 * (HMAG / 64) + 2;
constexpr int TILE_ZERO = 1 + HMAG / 64;

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

__device__ inline uint32_t as_u32(u16x2 v) { return __builtin_bit_cast(uint32_t, v); }
__device__ inline u16x2 as_u16x2(uint32_t v) { return __builtin_bit_cast(u16x2, v); }

// Two patterns less HLO; a half is inside the window exactly when its bits 12..14 are 0.
__device__ inline uint32_t window_words(uint32_t w)
{
    const u16x2 lo = {(unsigned short)HLO, (unsigned short)HLO};
    return as_u32(as_u16x2(w) - lo);
}
// bin * 4 of both halves: magnitude in bits 3..14, sign in bit 2
__device__ inline uint32_t bin_offsets(uint32_t t)
{
    const u16x2 v = as_u16x2(t), a = {3, 3}, b = {13, 13};
    return as_u32(v << a) | as_u32(v >> b);
}

__device__ inline float pattern_value(uint32_t p) { return __uint_as_float(p << 16); }
__device__ inline uint32_t vec_word(const uint4 &v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

struct CutLds {
    uint32_t count[NTILES];        // ids per tile
    uint32_t before[NTILES];       // ids in earlier tiles
    double sum[NTILES];            // kept weight per tile after top-k
    double sum_m[NTILES];          // of it the weights that pass min-p
    float xval[2][64];             // tiles 0 and 65: values, largest first
    uint32_t xcnt[2][64];
    uint32_t xlist[HX];            // patterns outside the window as they were met
    uint32_t nx, zeros, low, bad;  // how many; zeros; largest order key <= -2^8; NaN or +inf met
    int total, first;              // ids counted; first tile with any
    float max;
    RowCut cut;
};

__device__ inline void cut_lds_clear(CutLds &c)
{
    if (threadIdx.x == 0)
        c.nx = c.zeros = c.low = c.bad = 0;
}

// What a thread meets outside the window.
struct Outside {
    uint32_t zeros = 0, low = 0, bad = 0;
};

__device__ inline void count_outside(uint32_t p, CutLds &c, Outside &o)
{
    const uint32_t a = p & 0x7fffu;
    if (a == 0) {
        o.zeros++;
    } else if (a >= 0x7f80u) {
        o.bad |= p != 0xff80u;
    } else if ((p & 0x8000u) && a >= HLO) {
        o.low = max(o.low, order_key(pattern_value(p)));
    } else {
        const uint32_t i = atomicAdd(&c.nx, 1u);
        if (i < HX)
            c.xlist[i] = p;
    }
}

__device__ inline void count_one(uint32_t p, uint32_t *hist, CutLds &c, Outside &o)
{
    const uint32_t t = (p - HLO) & 0xffffu;
    if ((t & 0x7000u) == 0)
        atomicAdd(&hist[((t & 0xfffu) << 1) | (t >> 15)], 1u);
    else
        count_outside(p, c, o);
}

__device__ inline void bump(uint32_t *hist, uint32_t off)
{
    atomicAdd(reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(hist) + off), 1u);
}

// Counts eight patterns.  The common case, all lanes inside the window, takes seven VALU
// instructions for two patterns and one LDS add for each.
__device__ inline void count_vec(const uint4 &v, uint32_t *hist, CutLds &c, Outside &o)
{
    uint32_t t[4], out = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t[i] = window_words(vec_word(v, i));
        out |= t[i] & 0x70007000u;
    }
    if (__ballot(out != 0) == 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t b = bin_offsets(t[i]);
            bump(hist, b & 0xffffu);
            bump(hist, b >> 16);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            count_one(vec_word(v, i) & 0xffffu, hist, c, o);
            count_one(vec_word(v, i) >> 16, hist, c, o);
        }
    }
}

// A row as whole 16-byte vectors, with the ids before the first and after the last one by one.
struct RowSpan {
    const char *row;
    const uint4 *vec;
    int head, nvec, tail0;     // ids before vec; vectors; first id after them
};

__device__ inline RowSpan row_span(const char *row, int V)
{
    RowSpan r;
    r.row = row;
    const int mis = (int)(reinterpret_cast<uintptr_t>(row) & 15);
    r.head = min(V, mis ? (16 - mis) / 2 : 0);
    r.vec = reinterpret_cast<const uint4 *>(row + 2 * (size_t)r.head);
    r.nvec = (V - r.head) / 8;
    r.tail0 = r.head + r.nvec * 8;
    return r;
}

__device__ inline uint32_t pattern_at(const char *row, int id)
{
    return reinterpret_cast<const uint16_t *>(row)[id];
}

__device__ inline uint32_t wave_sum_u32(uint32_t v)
{
    int x = (int)v;
    x += lane_xch<0>(x);
    x += lane_xch<1>(x);
    x += lane_xch<2>(x);
    x += lane_xch<3>(x);
    x += lane_xch<4>(x);
    x += lane_xch<5>(x);
    return (uint32_t)x;
}

__device__ inline uint32_t wave_scan_u32(uint32_t v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const uint32_t u = (uint32_t)__shfl_up((int)v, o);
        if (lane >= o)
            v += u;
    }
    return v;
}

// A tile's lane: its value, its count, and its bin (-1 outside the window).
__device__ inline void tile_entry(int tile, const uint32_t *hist, const CutLds &c, float &x,
                                  uint32_t &n, int &bin)
{
    const int lane = threadIdx.x & 63;
    if (tile == 0 || tile == TILE_ZERO) {
        x = c.xval[tile != 0][lane];
        n = c.xcnt[tile != 0][lane];
        bin = -1;
        return;
    }
    const bool neg = tile > TILE_ZERO;
    const int mag = neg ? (tile - TILE_ZERO - 1) * 64 + lane : HMAG - 1 - ((tile - 1) * 64 + lane);
    bin = 2 * mag + (int)neg;
    n = hist[bin];
    x = pattern_value(HLO + (uint32_t)mag + (neg ? 0x8000u : 0u));
}

// The values kept apart, in order, into tiles 0 and 65 (wave 0).
__device__ inline void order_outside(CutLds &c)
{
    const int lane = threadIdx.x & 63;
    c.xcnt[0][lane] = c.xcnt[1][lane] = 0;
    c.xval[0][lane] = c.xval[1][lane] = 0.0f;
    const int n = (int)min(c.nx, (uint32_t)HX - 1);
    // lane n stands for the zeros
    const float x = lane < n ? pattern_value(c.xlist[lane]) : 0.0f;
    const uint32_t mine = lane < n ? 1u : lane == n ? c.zeros : 0u;
    const bool high = x >= 256.0f;
    if (n == 0) {
        if (lane == 0)
            c.xcnt[1][0] = c.zeros;
        return;
    }
    uint32_t cnt = 0;
    bool first = lane <= n;
    for (int j = 0; j <= n; ++j) {
        const float y = __shfl(x, j);
        const uint32_t m = (uint32_t)__shfl((int)mine, j);
        cnt += y == x ? m : 0u;
        first = first && !(y == x && j < lane);
    }
    const unsigned long long firsts = __ballot(first);
    int rank = 0;
    for (int j = 0; j <= n; ++j) {
        const float y = __shfl(x, j);
        rank += (firsts >> j & 1) && y > x && (y >= 256.0f) == high;
    }
    if (first) {
        c.xcnt[!high][rank] = cnt;
        c.xval[!high][rank] = x;
    }
}

// What top-k leaves of a tile's counts: nothing past the first k ids.
__device__ inline uint32_t clip_counts(uint32_t n, uint32_t before, uint32_t tile_count, int k)
{
    if (before >= (uint32_t)k)
        return 0;
    if (before + tile_count <= (uint32_t)k)
        return n;
    const uint32_t b = before + wave_scan_u32(n) - n;
    return b >= (uint32_t)k ? 0u : min(n, (uint32_t)k - b);
}

// The cut from the counts.  NW waves; on return c.cut holds the result for all.  With `table`,
// table[bin] receives the weight of every bin that occurs among the first k ids.
template <int NW>
__device__ void cut_from_counts(const uint32_t *hist, CutLds &c, const Outside &o, const Params &q,
                                int V, double *table)
{
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    if (o.zeros)
        atomicAdd(&c.zeros, o.zeros);
    if (o.low)
        atomicMax(&c.low, o.low);
    if (o.bad)
        atomicOr(&c.bad, 1u);
    __syncthreads();
    if (wv == 0)
        order_outside(c);
    __syncthreads();
    for (int t = wv; t < NTILES; t += NW) {
        float x;
        uint32_t n;
        int bin;
        tile_entry(t, hist, c, x, n, bin);
        const uint32_t s = __ballot(n != 0) ? wave_sum_u32(n) : 0u;
        if (lane == 0)
            c.count[t] = s;
    }
    __syncthreads();
    if (wv == 0) {
        // three tiles to a lane
        uint32_t a[3], s = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            a[i] = lane * 3 + i < NTILES ? c.count[lane * 3 + i] : 0u;
            s += a[i];
        }
        const uint32_t inc = wave_scan_u32(s);
        uint32_t b = inc - s;
        int first = NTILES;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            if (lane * 3 + i < NTILES)
                c.before[lane * 3 + i] = b;
            if (a[i] && first == NTILES)
                first = lane * 3 + i;
            b += a[i];
        }
        const unsigned long long any = __ballot(first != NTILES);
        const int t0 = any ? __shfl(first, __ffsll(any) - 1) : 0;
        float x;
        uint32_t n;
        int bin;
        tile_entry(t0, hist, c, x, n, bin);
        const unsigned long long has = __ballot(n != 0);
        x = __shfl(x, has ? __ffsll(has) - 1 : 0);
        const int total = __shfl((int)inc, 63);
        if (lane == 0) {
            c.total = total;
            c.first = t0;
            c.max = x;
            RowCut r;
            r.z = 0.0;
            r.c = q.c;
            r.max = x;
            r.cut = KEY_NEG_INF;
            r.tie = V;
            r.state = CUT_READY;
            if (!q.ok || c.bad || (total == 0 && c.low == 0)) {
                r.state = CUT_NONE;
            } else if (c.nx >= HX || total == 0) {
                r.state = CUT_EXACT;
            } else if (c.low) {
                // the low values count if one of them could be kept with a weight that matters
                const double w = weight(key_value(c.low), x, q.c);
                if (w > 0.0 && (w >= 0x1p-80 || (q.k < V && q.k > total) || (q.m > 0.0 && w >= q.m)))
                    r.state = CUT_EXACT;
            }
            c.cut = r;
        }
    }
    __syncthreads();
    if (c.cut.state != CUT_READY)
        return;
    const float M = c.max;
    const int total = c.total, k = min(q.k, total);
    for (int t = wv; t < NTILES; t += NW) {
        const uint32_t cnt = c.count[t], b = c.before[t];
        double s = 0.0, sm = 0.0;
        if (cnt && b < (uint32_t)k) {
            float x;
            uint32_t n;
            int bin;
            tile_entry(t, hist, c, x, n, bin);
            const uint32_t left = clip_counts(n, b, cnt, k);
            const double w = left ? weight(x, M, q.c) : 0.0;
            if (table && left && bin >= 0)
                table[bin] = w;
            s = wave_sum((double)left * w);
            sm = q.m > 0.0 ? wave_sum(w >= q.m ? (double)left * w : 0.0) : s;
        }
        if (lane == 0) {
            c.sum[t] = s;
            c.sum_m[t] = sm;
        }
    }
    __syncthreads();
    if (wv == 0) {
        double a[3], am[3], s = 0.0, sm = 0.0;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const bool in = lane * 3 + i < NTILES;
            a[i] = in ? c.sum[lane * 3 + i] : 0.0;
            am[i] = in ? c.sum_m[lane * 3 + i] : 0.0;
            s += a[i];
            sm += am[i];
        }
        const double inc = wave_incl_scan(s), before = wave_excl_from_incl(inc);
        const double zk = lane_value(inc, 63), zm = wave_sum(sm);
        // the tile of the cut and, in it, what comes before
        int tile = -1;
        double base = 0.0;
        const double goal = q.p < 1.0 ? q.p * zk : INFINITY;
        if (q.p < 1.0 || k < total) {
            double b = before;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const int t = lane * 3 + i;
                if (t < NTILES && c.count[t] && c.before[t] < (uint32_t)k && (b < goal || t == c.first)) {
                    tile = t;
                    base = b;
                }
                b += a[i];
            }
            const unsigned long long has = __ballot(tile >= 0);
            const int l = 63 - __clzll(has);
            tile = __shfl(tile, l);
            base = lane_value(base, l);
        }
        RowCut r = c.cut;
        r.z = zk;
        double wcut = 0.0;
        if (tile >= 0) {
            float x;
            uint32_t n;
            int bin;
            tile_entry(tile, hist, c, x, n, bin);
            const uint32_t left = clip_counts(n, c.before[tile], c.count[tile], k);
            const double w = left ? weight(x, M, q.c) : 0.0;
            const double in = wave_incl_scan((double)left * w);
            const double bef = base + wave_excl_from_incl(in);
            unsigned long long has = __ballot(left && bef < goal);
            if (!has)
                has = __ballot(left != 0) & -__ballot(left != 0);   // p = 0: the first alone
            const int l = 63 - __clzll(has);
            const double bl = lane_value(bef, l), wl = lane_value(w, l);
            const uint32_t nl = (uint32_t)__shfl((int)n, l), ll = (uint32_t)__shfl((int)left, l);
            uint32_t keep = ll;
            if (q.p < 1.0) {
                const double m = ceil((goal - bl) / wl);
                keep = m < 1.0 ? 1u : m > (double)ll ? ll : (uint32_t)m;
            }
            wcut = wl;
            r.cut = order_key(__shfl(x, l));
            r.z = q.p < 1.0 ? bl + (double)keep * wl : zk;
            r.state = keep < nl ? CUT_TIES : CUT_READY;
            r.tie = keep < nl ? (int)keep : V;
        }
        if (q.m > 0.0 && wcut < q.m) {
            // min-p is the tighter: the last value that passes it
            int mt = -1;
#pragma unroll
            for (int i = 0; i < 3; ++i)
                if (am[i] > 0.0)
                    mt = lane * 3 + i;
            const int l = 63 - __clzll(__ballot(mt >= 0));
            mt = __shfl(mt, l);
            float x;
            uint32_t n;
            int bin;
            tile_entry(mt, hist, c, x, n, bin);
            const uint32_t left = clip_counts(n, c.before[mt], c.count[mt], k);
            const double w = left ? weight(x, M, q.c) : 0.0;
            const unsigned long long has = __ballot(left && w >= q.m);
            const int ll = 63 - __clzll(has);
            const uint32_t nl = (uint32_t)__shfl((int)n, ll), fl = (uint32_t)__shfl((int)left, ll);
            r.cut = order_key(__shfl(x, ll));
            r.z = zm;
            r.state = fl < nl ? CUT_TIES : CUT_READY;
            r.tie = fl < nl ? (int)fl : V;
        }
        if (lane == 0)
            c.cut = r;
    }
    __syncthreads();
}

// Counts a whole row straight from memory, eight vectors of a thread in flight.
template <int WGT>
__device__ void count_row(const RowSpan &r, int V, uint32_t *hist, CutLds &c, Outside &o)
{
    const int t = threadIdx.x;
    constexpr int U = 4;
    uint4 v[U];
    int i = t;
    if (i + (U - 1) * WGT < r.nvec) {
#pragma unroll
        for (int k = 0; k < U; ++k)
            v[k] = load_stream(reinterpret_cast<const char *>(r.vec + i + k * WGT));
        i += U * WGT;
        for (; i + (U - 1) * WGT < r.nvec; i += U * WGT) {
            uint4 nx[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                nx[k] = load_stream(reinterpret_cast<const char *>(r.vec + i + k * WGT));
#pragma unroll
            for (int k = 0; k < U; ++k)
                count_vec(v[k], hist, c, o);
#pragma unroll
            for (int k = 0; k < U; ++k)
                v[k] = nx[k];
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            count_vec(v[k], hist, c, o);
    }
    for (; i < r.nvec; i += WGT)
        count_vec(load_stream(reinterpret_cast<const char *>(r.vec + i)), hist, c, o);
    if (t < r.head)
        count_one(pattern_at(r.row, t), hist, c, o);
    if (r.tail0 + t < V)
        count_one(pattern_at(r.row, r.tail0 + t), hist, c, o);
}

template <int WGT> __device__ void clear_hist(uint32_t *hist)
{
    for (int i = threadIdx.x; i < HBINS / 4; i += WGT)
        reinterpret_cast<uint4 *>(hist)[i] = make_uint4(0, 0, 0, 0);
}

constexpr int RWG = 512;   // threads per row of a bfloat16 verify: four workgroups to a compute unit

// The RowCut of every target and draft row of a bfloat16 verify.
__global__ __launch_bounds__(RWG, 8) void k_filter_rows_bf16(const char *tgt, const char *drf, int B,
                                                             int K, int V, FilterPtrs ft,
                                                             FilterPtrs fd, RowCut *cuts)
{
    __shared__ __align__(16) uint32_t hist[HBINS];
    __shared__ CutLds c;
    const int n = blockIdx.x, nt = B * (K + 1);
    const bool is_t = n < nt;
    const char *row = (is_t ? tgt + (size_t)n * V * 2 : drf + (size_t)(n - nt) * V * 2);
    const Params q = is_t ? load_params(ft, n / (K + 1), V) : load_params(fd, (n - nt) / K, V);
    clear_hist<RWG>(hist);
    cut_lds_clear(c);
    __syncthreads();
    Outside o;
    count_row<RWG>(row_span(row, V), V, hist, c, o);
    cut_from_counts<RWG / 64>(hist, c, o, q, V, nullptr);
    if (threadIdx.x == 0)
        cuts[n] = c.cut;
}

// ------------------------------------------------------------------ the inverse-CDF draw
//
// A row is read in groups of one 16-byte vector, group 0 being the ids before the first aligned
// vector and the last group those after the last whole one.  Each of a workgroup's waves takes a
// contiguous range of groups, 64 at a time (a unit); a unit's kept weight is summed in a fixed
// order and noted in LDS.  The draw then finds the wave, the unit, the lane and the id whose
// cumulative weight passes u * total, reading again only that unit.

template <int DT> struct Groups {
    static constexpr int E = Elt<DT>::EPV;
    const char *row;
    int V, head, count, per_wave;      // ids before the first vector; groups; units per wave

    __device__ Groups(const char *r, int v) : row(r), V(v)
    {
        const int mis = (int)(reinterpret_cast<uintptr_t>(r) & 15);
        head = min(v, mis ? (16 - mis) / Elt<DT>::BYTES : 0);
        count = (v - head) / E + 2;
        per_wave = (count + FWAVES * 64 - 1) / (FWAVES * 64);
    }
    __device__ int first_id(int g) const { return head + (g - 1) * E; }
    __device__ int group_of(int wave, int unit, int lane) const
    {
        return (wave * per_wave + unit) * 64 + lane;
    }
    // the group's logits; -inf where it has no id
    __device__ uint4 load(int g) const
    {
        if (g > 0 && g < count - 1)
            return load_plain(row + (ptrdiff_t)first_id(g) * Elt<DT>::BYTES);
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = DT == 1 ? 0xff80ff80u : 0xff800000u;
        if (g == 0 || g == count - 1) {
            const int i0 = first_id(g), end = g == 0 ? head : V;
#pragma unroll
            for (int k = 0; k < E; ++k) {
                if (i0 + k < 0 || i0 + k >= end)
                    continue;
                if constexpr (DT == 1) {
                    const uint32_t p = pattern_at(row, i0 + k);
                    w[k / 2] = k & 1 ? (w[k / 2] & 0xffffu) | p << 16 : (w[k / 2] & 0xffff0000u) | p;
                } else {
                    w[k] = __float_as_uint(Elt<DT>::one(row, i0 + k));
                }
            }
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

constexpr int MAX_UNITS_BF16 = (MAX_VOCAB / 8 + 2 + 63) / 64 + FWAVES;
constexpr int MAX_UNITS_F32 = (MAX_VOCAB / 4 + 2 + 63) / 64 + FWAVES;
template <int DT> constexpr int max_units() { return DT == 1 ? MAX_UNITS_BF16 : MAX_UNITS_F32; }

struct DrawLds {
    double wave[FWAVES];
    uint32_t ties[FWAVES];
    int id;
};

// units[w * per_wave + i] hold the sums of all units (written by their waves); weights(g, vec, x)
// gives the E weights of a group.  Returns the drawn id in every thread, -1 if all weights are 0.
template <int DT, typename W>
__device__ int draw_from_units(const Groups<DT> &gr, const double *units, double u, DrawLds &lds,
                               W weights)
{
    constexpr int E = Elt<DT>::EPV;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const double *mine = units + wv * gr.per_wave;
    double s = 0.0;
    for (int i = lane; i < gr.per_wave; i += 64)
        s += mine[i];
    s = wave_sum(s);
    if (lane == 0)
        lds.wave[wv] = s;
    if (threadIdx.x == 0)
        lds.id = -1;
    __syncthreads();
    double total = 0.0;
    for (int i = 0; i < FWAVES; ++i)
        total += lds.wave[i];
    double goal = u * total;
    int pick = -1;
    double base = 0.0, run = 0.0;
    for (int i = 0; i < FWAVES; ++i) {
        const double x = lds.wave[i];
        if (x > 0.0) {
            pick = i;
            base = run;
            run += x;
            if (run > goal)
                break;
        }
    }
    if (wv == pick) {
        int unit = -1, last = 0;
        for (int i0 = 0; i0 < gr.per_wave && unit < 0; i0 += 64) {
            const double x = i0 + lane < gr.per_wave ? mine[i0 + lane] : 0.0;
            const double inc = wave_incl_scan(x), exc = wave_excl_from_incl(inc);
            const unsigned long long pos = __ballot(x > 0.0);
            const unsigned long long over = __ballot(x > 0.0 && base + inc > goal);
            if (over) {
                const int l = __ffsll(over) - 1;
                unit = i0 + l;
                base += lane_value(exc, l);
            } else {
                if (pos)
                    last = i0 + 63 - __clzll(pos);
                base += lane_value(inc, 63);
            }
        }
        if (unit < 0) {                      // rounding left none: the last id of positive weight
            unit = last;
            goal = INFINITY;
        }
        const int g = gr.group_of(wv, unit, lane);
        double x[E], sum = 0.0;
        weights(g, gr.load(g), x);
#pragma unroll
        for (int k = 0; k < E; ++k)
            sum += x[k];
        const double inc = wave_incl_scan(sum), before = base + wave_excl_from_incl(inc);
        const unsigned long long pos = __ballot(sum > 0.0);
        const unsigned long long over = __ballot(sum > 0.0 && base + inc > goal);
        const int l = over ? __ffsll(over) - 1 : 63 - __clzll(pos);
        if (lane == l) {
            int id = -1;
            double r = before;
#pragma unroll
            for (int k = 0; k < E; ++k) {
                if (x[k] > 0.0 && !(id >= 0 && r > goal)) {
                    r += x[k];
                    id = gr.first_id(g) + k;
                }
            }
            lds.id = id;
        }
    }
    __syncthreads();
    return lds.id;
}

// Sums the kept weight of each of the wave's units; vec(i, g) is unit i's group g.
template <int DT, typename V, typename A, typename W>
__device__ void sum_unit(const Groups<DT> &gr, int i, double *units, V vec, A any, W weights)
{
    constexpr int E = Elt<DT>::EPV;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    double s = 0.0;
    if (__ballot(any(vec)) != 0) {
        double x[E];
        weights(gr.group_of(wv, i, lane), vec, x);
#pragma unroll
        for (int k = 0; k < E; ++k)
            s += x[k];
        s = wave_sum(s);
    }
    if (lane == 0)
        units[wv * gr.per_wave + i] = s;
}

// The last kept id among those equal to the cut, the n-th of them: equals per unit, then the wave,
// the unit, the lane and the id.
template <int DT, typename F>
__device__ int nth_equal(const Groups<DT> &gr, uint32_t cut, int n, uint32_t *units, DrawLds &lds,
                         F vec)
{
    constexpr int E = Elt<DT>::EPV;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    auto equals = [&](const uint4 &v) {
        float x[E];
        Elt<DT>::unpack(v, x);
        const float y = key_value(cut);
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < E; ++k)
            m |= (uint32_t)(x[k] == y) << k;
        return m;
    };
    uint32_t all = 0;
    for (int i = 0; i < gr.per_wave; ++i) {
        const uint32_t m = equals(vec(i));
        const uint32_t s = __ballot(m != 0) ? wave_sum_u32(__popc(m)) : 0u;
        if (lane == 0)
            units[wv * gr.per_wave + i] = s;
        all += s;
    }
    if (lane == 0)
        lds.ties[wv] = all;
    if (threadIdx.x == 0)
        lds.id = 0x7fffffff;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < wv; ++w)
        before += (int)lds.ties[w];
    if (before < n && n <= before + (int)all) {
        const uint32_t *mine = units + wv * gr.per_wave;
        int unit = -1;
        for (int i0 = 0; i0 < gr.per_wave && unit < 0; i0 += 64) {
            const int x = i0 + lane < gr.per_wave ? (int)mine[i0 + lane] : 0;
            const int inc = (int)wave_scan_u32((uint32_t)x);
            const unsigned long long here = __ballot(before + inc >= n);
            if (here) {
                const int l = __ffsll(here) - 1;
                unit = i0 + l;
                before += __shfl(inc - x, l);
            } else {
                before += __shfl(inc, 63);
            }
        }
        const int g = gr.group_of(wv, unit, lane);
        uint32_t m = equals(gr.load(g));
        const int c = __popc(m), b = before + (int)wave_scan_u32((uint32_t)c) - c;
        if (b < n && n <= b + c) {
            for (int skip = n - b - 1; skip > 0; --skip)
                m &= m - 1;
            lds.id = gr.first_id(g) + __ffs(m) - 1;
        }
    }
    __syncthreads();
    return lds.id;
}

// Weights of a group under a cut law, computed from the logits: w / z.
template <int DT> struct DirectLaw {
    const Groups<DT> &gr;
    const RowCut &r;
    double z;
    __device__ void operator()(int g, const uint4 &v, double (&x)[Elt<DT>::EPV]) const
    {
        float y[Elt<DT>::EPV];
        Elt<DT>::unpack(v, y);
#pragma unroll
        for (int k = 0; k < Elt<DT>::EPV; ++k) {
            x[k] = 0.0;
            if (kept(order_key(y[k]), gr.first_id(g) + k, r) && y[k] != -INFINITY)
                x[k] = weight(y[k], r.max, r.c) / z;
        }
    }
};

// The same from a table of w / z by bin, 0 for what the cut leaves out.
struct TableLaw {
    const Groups<1> &gr;
    const RowCut &r;
    double z;
    const double *table;
    __device__ double at(uint32_t off) const
    {
        return *reinterpret_cast<const double *>(reinterpret_cast<const char *>(table) + 2 * off);
    }
    __device__ double one(uint32_t p, int id) const
    {
        const uint32_t t = (p - HLO) & 0xffffu;
        const float y = pattern_value(p);
        if ((t & 0x7000u) == 0) {
            const double w = table[((t & 0xfffu) << 1) | (t >> 15)];
            return order_key(y) == r.cut && id > r.tie ? 0.0 : w;
        }
        if ((p & 0x7fffu) >= 0x7f80u || !kept(order_key(y), id, r))
            return 0.0;
        return weight(y, r.max, r.c) / z;
    }
    __device__ void operator()(int g, const uint4 &v, double (&x)[8]) const
    {
        uint32_t t[4], out = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t[i] = window_words(vec_word(v, i));
            out |= t[i] & 0x70007000u;
        }
        // ids past the last kept tie are looked at one by one only where a tie may be among them
        if (__ballot(out != 0 || gr.first_id(g) + 7 > r.tie) == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t b = bin_offsets(t[i]);
                x[2 * i] = at(b & 0xffffu);
                x[2 * i + 1] = at(b >> 16);
            }
        } else {
            const int id = gr.first_id(g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = one(vec_word(v, i) & 0xffffu, id + 2 * i);
                x[2 * i + 1] = one(vec_word(v, i) >> 16, id + 2 * i + 1);
            }
        }
    }
};

// Whether a group can hold a kept id.  For a cut above zero patterns compare as signed 16-bit
// integers, two at a time.
template <int DT> struct MayKeep {
    uint32_t below;      // the largest pattern, twice, below the cut; 0: any group may
    __device__ explicit MayKeep(const RowCut &r)
    {
        const float y = key_value(r.cut);
        below = 0;
        if (DT == 1 && y > 0.0f)
            below = ((__float_as_uint(y) >> 16) - 1) * 0x10001u;
    }
    __device__ bool operator()(const uint4 &v) const
    {
        if (DT != 1 || below == 0)
            return true;
        typedef short s16x2 __attribute__((ext_vector_type(2)));
        const s16x2 b = __builtin_bit_cast(s16x2, below);
        uint32_t d = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            d |= __builtin_bit_cast(uint32_t, __builtin_elementwise_max(
                     __builtin_bit_cast(s16x2, vec_word(v, i)), b)) ^ below;
        return d != 0;
    }
};

// table[bin] = w / z for the bins that r keeps, 0 for the others.
__device__ void fill_table(const RowCut &r, double *table)
{
    for (int b = threadIdx.x; b < HBINS; b += FWG) {
        const float x = pattern_value(HLO + (uint32_t)(b >> 1) + (b & 1 ? 0x8000u : 0u));
        table[b] = order_key(x) >= r.cut && x <= r.max ? weight(x, r.max, r.c) / r.z : 0.0;
    }
}

constexpr int RES = 16;    // vectors of its row that a thread keeps in registers: 131072 ids

// One row: its cut by counting, then the draw from the same registers.
__global__ __launch_bounds__(FWG, 4) void k_filter_sample_bf16(const char *logits, int V,
                                                               int64_t stride, FilterPtrs f,
                                                               const float *unif, int *tok,
                                                               float *prob)
{
    __shared__ __align__(16) uint32_t hist[HBINS];
    __shared__ double table[HBINS];
    __shared__ CutLds c;
    __shared__ DrawLds dl;
    __shared__ RedLds red;
    double *units = reinterpret_cast<double *>(hist);
    static_assert(sizeof(hist) >= MAX_UNITS_BF16 * sizeof(double), "units fit where the counts were");
    const int n = blockIdx.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const char *row = logits + (size_t)n * stride * 2;
    const Groups<1> gr(row, V);
    uint4 v[RES];
#pragma unroll
    for (int i = 0; i < RES; ++i)
        if (i < gr.per_wave)
            v[i] = gr.load(gr.group_of(wv, i, lane));
    const Params q = load_params(f, n, V);
    clear_hist<FWG>(hist);
    cut_lds_clear(c);
    __syncthreads();
    Outside o;
#pragma unroll
    for (int i = 0; i < RES; ++i)
        if (i < gr.per_wave)
            count_vec(v[i], hist, c, o);
    for (int i = RES; i < gr.per_wave; ++i)
        count_vec(gr.load(gr.group_of(wv, i, lane)), hist, c, o);
    cut_from_counts<FWAVES>(hist, c, o, q, V, table);
    RowCut r = c.cut;
    const bool counted = r.state != CUT_EXACT;
    if (!counted)
        r = cut_by_bisection<1>(row, V, q, red);
    if (r.state == CUT_NONE) {
        if (threadIdx.x == 0) {
            tok[n] = -1;
            if (prob)
                prob[n] = NAN;
        }
        return;
    }
    auto held = [&](int i) { return gr.load(gr.group_of(wv, i, lane)); };
    if (r.state == CUT_TIES) {
        r.tie = nth_equal(gr, r.cut, r.tie, reinterpret_cast<uint32_t *>(hist), dl, held);
        __syncthreads();
    }
    const MayKeep<1> may(r);
    int id;
    if (counted) {
        // the table holds the weights of the bins that occur; those below the cut go to 0
        for (int b = threadIdx.x; b < HBINS; b += FWG)
            if (order_key(pattern_value(HLO + (uint32_t)(b >> 1) + (b & 1 ? 0x8000u : 0u))) < r.cut)
                table[b] = 0.0;
        __syncthreads();
        const TableLaw law{gr, r, 1.0, table};
#pragma unroll
        for (int i = 0; i < RES; ++i)
            if (i < gr.per_wave)
                sum_unit(gr, i, units, v[i], may, law);
        for (int i = RES; i < gr.per_wave; ++i)
            sum_unit(gr, i, units, held(i), may, law);
        __syncthreads();
        id = draw_from_units(gr, units, (double)unif[n], dl, law);
    } else {
        const DirectLaw<1> law{gr, r, 1.0};
        for (int i = 0; i < gr.per_wave; ++i)
            sum_unit(gr, i, units, held(i), may, law);
        __syncthreads();
        id = draw_from_units(gr, units, (double)unif[n], dl, law);
    }
    if (threadIdx.x == 0) {
        tok[n] = id;
        if (prob)
            prob[n] = id < 0 ? NAN : (float)(weight(Elt<1>::one(row, id), r.max, r.c) / r.z);
    }
}

__global__ __launch_bounds__(FWG) void k_filter_sample_f32(const char *logits, int V, int64_t stride,
                                                           FilterPtrs f, const float *unif, int *tok,
                                                           float *prob)
{
    __shared__ RedLds red;
    __shared__ DrawLds dl;
    __shared__ double units[MAX_UNITS_F32];
    const int n = blockIdx.x, lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const char *row = logits + (size_t)n * stride * 4;
    const RowCut r = cut_by_bisection<0>(row, V, load_params(f, n, V), red);
    int id = -1;
    if (r.state == CUT_READY) {
        const Groups<0> gr(row, V);
        const MayKeep<0> may(r);
        const DirectLaw<0> law{gr, r, 1.0};
        for (int i = 0; i < gr.per_wave; ++i)
            sum_unit(gr, i, units, gr.load(gr.group_of(wv, i, lane)), may, law);
        __syncthreads();
        id = draw_from_units(gr, units, (double)unif[n], dl, law);
    }
    if (threadIdx.x == 0) {
        tok[n] = id;
        if (prob)
            prob[n] = id < 0 ? NAN : (float)(weight(Elt<0>::one(row, id), r.max, r.c) / r.z);
    }
}

// The RowCut of every target and draft row of a float32 verify: the B (K+1) target rows, then the
// B K draft rows.
__global__ __launch_bounds__(FWG) void k_filter_rows_f32(const char *tgt, const char *drf, int B,
                                                         int K, int V, FilterPtrs ft, FilterPtrs fd,
                                                         RowCut *cuts)
{
    __shared__ RedLds red;
    const int n = blockIdx.x, nt = B * (K + 1);
    const bool is_t = n < nt;
    const char *row = is_t ? tgt + (size_t)n * V * 4 : drf + (size_t)(n - nt) * V * 4;
    const Params q = is_t ? load_params(ft, n / (K + 1), V) : load_params(fd, (n - nt) / K, V);
    const RowCut r = cut_by_bisection<0>(row, V, q, red);
    if (threadIdx.x == 0)
        cuts[n] = r;
}

// The law's value at one id.
template <int DT>
__device__ inline double law_at(const char *row, int id, const RowCut &r)
{
    const float x = Elt<DT>::one(row, id);
    return kept(order_key(x), id, r) ? weight(x, r.max, r.c) / r.z : 0.0;
}

constexpr int MAX_POS = 63;

struct VerifyLds {
    RowCut cut[2 * MAX_POS + 1];      // target rows 0..K, then draft rows 0..K-1
    double P[MAX_POS + 1], Q[MAX_POS + 1];
    int L;
    unsigned long long look;
};

// Accept tests, first rejection and the replacement or bonus draw of one sequence.
template <int DT>
__global__ __launch_bounds__(FWG, 4) void k_filter_verify(const char *tgt, const char *drf, int B,
                                                          int K, int V, FilterPtrs ft, FilterPtrs fd,
                                                          const int *tokens, const float *unif,
                                                          const RowCut *cuts, int *acc, int *out,
                                                          float *probs)
{
    constexpr int E = Elt<DT>::EPV;
    __shared__ double tables[DT == 1 ? 2 : 1][DT == 1 ? HBINS : 1];
    __shared__ double units[max_units<DT>()];
    __shared__ VerifyLds s;
    __shared__ DrawLds dl;
    __shared__ RedLds red;
    const int b = blockIdx.x, t = threadIdx.x, lane = t & 63, wv = t >> 6;
    const size_t rb = (size_t)V * Elt<DT>::BYTES;
    const char *trow = tgt + (size_t)b * (K + 1) * rb, *drow = drf + (size_t)b * K * rb;
    auto row_of = [&](int i) { return i <= K ? trow + i * rb : drow + (i - K - 1) * rb; };
    if (t < 2 * K + 1)
        s.cut[t] = t <= K ? cuts[(size_t)b * (K + 1) + t]
                          : cuts[(size_t)B * (K + 1) + (size_t)b * K + (t - K - 1)];
    __syncthreads();
    if (DT == 1)
        for (int i = 0; i < 2 * K + 1; ++i)
            if (s.cut[i].state == CUT_EXACT) {
                const RowCut r = cut_by_bisection<DT>(row_of(i), V, load_params(i <= K ? ft : fd, b, V), red);
                __syncthreads();
                if (t == 0)
                    s.cut[i] = r;
                __syncthreads();
            }
    // lane j: position j.  A draft id equal to a cut that keeps some of its ties is looked up
    // below; until then it counts as kept.
    if (t < 64) {
        bool ok = t <= K ? s.cut[t].state != CUT_NONE : true;
        bool lookp = false, lookq = false;
        double P = 0.0, Q = 0.0;
        if (t < K) {
            const int x = tokens[(size_t)b * K + t];
            const RowCut rp = s.cut[t], rq = s.cut[K + 1 + t];
            ok = ok && rq.state != CUT_NONE && x >= 0 && x < V;
            if (ok) {
                const float xp = Elt<DT>::one(trow + t * rb, x), xq = Elt<DT>::one(drow + t * rb, x);
                const uint32_t kp = order_key(xp), kq = order_key(xq);
                lookp = kp == rp.cut && rp.state == CUT_TIES;
                lookq = kq == rq.cut && rq.state == CUT_TIES;
                P = lookp || kept(kp, x, rp) ? weight(xp, rp.max, rp.c) / rp.z : 0.0;
                Q = lookq || kept(kq, x, rq) ? weight(xq, rq.max, rq.c) / rq.z : 0.0;
            }
            s.P[t] = P;
            s.Q[t] = Q;
        }
        const bool good = __ballot(!ok) == 0;
        const unsigned long long lp = __ballot(good && lookp), lq = __ballot(good && lookq);
        if (t == 0) {
            s.L = good ? 0 : -1;
            s.look = lp;
            dl.wave[0] = __longlong_as_double((long long)lq);
        }
    }
    __syncthreads();
    const unsigned long long lp = s.look, lq = (unsigned long long)__double_as_longlong(dl.wave[0]);
    __syncthreads();
    for (int i = 0; i < 2 * K + 1; ++i) {
        const bool is_t = i < K;
        const int j = is_t ? i : i - K - 1;
        if (i == K || !((is_t ? lp : lq) >> j & 1))
            continue;
        // how many ids below the draft's equal the cut
        const char *row = row_of(i);
        const int x = tokens[(size_t)b * K + j];
        const float y = key_value(s.cut[i].cut);
        int n = 0;
        for (int id = t; id < x; id += FWG)
            n += Elt<DT>::one(row, id) == y;
        n = block_sum(n, red.i);
        if (t == 0 && n >= s.cut[i].tie)
            (is_t ? s.P : s.Q)[j] = 0.0;
    }
    __syncthreads();
    if (t < 64) {
        const bool good = s.L >= 0;
        const double P = t < K ? s.P[t] : 0.0, Q = t < K ? s.Q[t] : 0.0;
        const bool take = t < K && P > 0.0 && (double)unif[(size_t)b * (K + 1) + t] * Q <= P;
        const unsigned long long rej = __ballot(t < K && !take);
        if (t < K && probs) {
            probs[((size_t)b * K + t) * 2] = good ? (float)P : NAN;
            probs[((size_t)b * K + t) * 2 + 1] = good ? (float)Q : NAN;
        }
        if (t == 0 && good)
            s.L = rej ? __ffsll(rej) - 1 : K;
    }
    __syncthreads();
    const int L = s.L;
    int id = -1;
    if (L >= 0) {
        const Groups<DT> gp(row_of(L), V);
        RowCut rp = s.cut[L], rq = rp;
        auto vp = [&](int i) { return gp.load(gp.group_of(wv, i, lane)); };
        uint32_t *counts = reinterpret_cast<uint32_t *>(units);
        if (rp.state == CUT_TIES) {
            rp.tie = nth_equal(gp, rp.cut, rp.tie, counts, dl, vp);
            __syncthreads();
        }
        const double u = (double)unif[(size_t)b * (K + 1) + K];
        const MayKeep<DT> may(rp);
        if constexpr (DT == 1)
            fill_table(rp, tables[0]);
        auto draw = [&](auto &weights) {
            for (int i = 0; i < gp.per_wave; ++i)
                sum_unit(gp, i, units, vp(i), may, weights);
            __syncthreads();
            return draw_from_units(gp, units, u, dl, weights);
        };
        auto with_law = [&](auto &p) {
            if (L < K) {
                const Groups<DT> gq(row_of(K + 1 + L), V);
                rq = s.cut[K + 1 + L];
                if (rq.state == CUT_TIES) {
                    rq.tie = nth_equal(gq, rq.cut, rq.tie, counts, dl,
                                       [&](int i) { return gq.load(gq.group_of(wv, i, lane)); });
                    __syncthreads();
                }
                if constexpr (DT == 1)
                    fill_table(rq, tables[1]);
                __syncthreads();
                // max(0, p - q); q is looked at only where p > 0
                auto residual = [&](int g, const uint4 &v, double (&x)[E]) {
                    p(g, v, x);
#pragma unroll
                    for (int k = 0; k < E; ++k)
                        if (x[k] > 0.0) {
                            const int i = gp.first_id(g) + k;
                            double y;
                            if constexpr (DT == 1)
                                y = TableLaw{gq, rq, rq.z, tables[DT == 1]}.one(pattern_at(gq.row, i), i);
                            else
                                y = law_at<DT>(gq.row, i, rq);
                            x[k] = fmax(x[k] - y, 0.0);
                        }
                };
                id = draw(residual);
                __syncthreads();
            }
            __syncthreads();
            if (id < 0)                     // the bonus draw, or nothing left of p - q
                id = draw(p);
        };
        if constexpr (DT == 1) {
            TableLaw p{gp, rp, rp.z, tables[0]};
            with_law(p);
        } else {
            DirectLaw<DT> p{gp, rp, rp.z};
            with_law(p);
        }
    }
    if (t <= K) {
        const size_t o = (size_t)b * (K + 1) + t;
        out[o] = t < L ? tokens[(size_t)b * K + t] : t == L ? id : -1;
    }
    if (t == 0)
        acc[b] = L;
}

}  // namespace

hipError_t launch_filter_sample(const Launch &ln, int dtype, int N, int V, int64_t stride,
                                const FilterPtrs &f, const void *logits, const float *unif,
                                int32_t *tok, float *prob)
{
    const char *x = static_cast<const char *>(logits);
    if (dtype == 1)
        SV_LAUNCH(ln, KIND_TAIL, k_filter_sample_bf16, dim3(N), dim3(FWG), 0, x, V, stride, f, unif,
                  tok, prob);
    else
        SV_LAUNCH(ln, KIND_TAIL, k_filter_sample_f32, dim3(N), dim3(FWG), 0, x, V, stride, f, unif,
                  tok, prob);
    return hipGetLastError();
}

template <int DT>
static hipError_t verify_impl(const Launch &ln, const Workspace &ws, int B, int K, int V,
                              const FilterPtrs &ft, const FilterPtrs &fd, const void *tgt,
                              const void *drf, const int32_t *tokens, const float *unif,
                              int32_t *acc, int32_t *out, float *probs)
{
    const char *t = static_cast<const char *>(tgt), *d = static_cast<const char *>(drf);
    RowCut *cuts = reinterpret_cast<RowCut *>(ws.part);
    const dim3 rows((unsigned)B * (2 * K + 1));
    if constexpr (DT == 1)
        SV_LAUNCH(ln, KIND_STATS, k_filter_rows_bf16, rows, dim3(RWG), 0, t, d, B, K, V, ft, fd, cuts);
    else
        SV_LAUNCH(ln, KIND_STATS, k_filter_rows_f32, rows, dim3(FWG), 0, t, d, B, K, V, ft, fd, cuts);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    SV_LAUNCH(ln, KIND_TAIL, k_filter_verify<DT>, dim3(B), dim3(FWG), 0, t, d, B, K, V, ft, fd,
              tokens, unif, cuts, acc, out, probs);
    return hipGetLastError();
}

hipError_t launch_filter_verify(const Launch &ln, const Workspace &ws, int dtype, int B, int K,
                                int V, const FilterPtrs &ft, const FilterPtrs &fd, const void *tgt,
                                const void *drf, const int32_t *tokens, const float *unif,
                                int32_t *acc, int32_t *out, float *probs)
{
    return (dtype == 1 ? verify_impl<1> : verify_impl<0>)(ln, ws, B, K, V, ft, fd, tgt, drf, tokens,
                                                          unif, acc, out, probs);
}

}  // namespace sv
