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
//   k_filter_sample_bf16, _f32   one 1024-thread workgroup per row: its RowCut, then the
//                                inverse-CDF draw; a decode step has a row per sequence, so this
//                                fills the chip with one launch
//   k_filter_rows_bf16, _f32     the RowCut of every target and draft row of a verify
//   k_filter_verify              one workgroup per sequence: accept tests, first rejection and
//                                the draw from p or from max(0, p - q)
//
// Ids are compared for equality with the definition, so weights and sums are fp64: sums good to
// 2^-24 would leave a draw's goal within their error of some id's edge in one of about 65 rows of
// 128256 (128256 edges, 2^-23 wide).  The one place with less, the integer sums of float32 top-p,
// says there what it loses.
//
// A row has to be read once; everything else here serves to keep the second look at it small.
// Counting patterns turns the cuts into arithmetic on 8192 bins instead of passes over the row
// (a bisection over values, the first kernels here, took 32 passes: 2929 us for 256 rows of
// 128256 where counting takes 43).
#include <float.h>

#include <type_traits>

#include "sv_device.h"
#include "sv_internal.h"

namespace sv {

namespace {

// f(0), ..., f(N - 1) with constant arguments: arrays indexed by them stay in registers.
template <int I, int N, typename F> __device__ __forceinline__ void unroll(F &&f)
{
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unroll<I + 1, N>(f);
    }
}
#define SV_INLINE __attribute__((always_inline))

constexpr int FWG = FILTER_WG;
constexpr int FWAVES = FWG / 64;

// Order-preserving 32-bit key of a logit: larger value, larger key; -0 and +0 are one key.
__device__ __forceinline__ uint32_t order_key(float x)
{
    const uint32_t u = __float_as_uint(x == 0.0f ? 0.0f : x);
    return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

constexpr uint32_t KEY_POS_INF = 0xff800000u;   // order_key(+inf); NaNs lie above it
constexpr uint32_t KEY_NEG_INF = 0x007fffffu;   // order_key(-inf); negative NaNs lie below it

// 2^a for a <= 0, within 2^-51: a = n + r with |r| <= 1/2, the Taylor polynomial of 2^r to r^13
// (whose rest is below (ln 2 / 2)^14 / 14! = 2^-57), scaled by 2^n.  Half the instructions of the
// general function, which every term of every sum would pay; 0 at and below 2^-1100.
__device__ __forceinline__ double exp2_neg(double a)
{
    a = fmax(a, -1100.0);
    const double n = rint(a), r = a - n;
    double p = 1.3691488853904128881e-12;
    p = fma(p, r, 2.5678435993488205142e-11);
    p = fma(p, r, 4.4455382718708114976e-10);
    p = fma(p, r, 7.0549116208011233299e-09);
    p = fma(p, r, 1.0178086009239699728e-07);
    p = fma(p, r, 1.3215486790144309488e-06);
    p = fma(p, r, 1.5252733804059840280e-05);
    p = fma(p, r, 1.5403530393381609954e-04);
    p = fma(p, r, 1.3333558146428443423e-03);
    p = fma(p, r, 9.6181291076284771620e-03);
    p = fma(p, r, 5.5504108664821579953e-02);
    p = fma(p, r, 2.4022650695910071233e-01);
    p = fma(p, r, 6.9314718055994530942e-01);
    p = fma(p, r, 1.0);
    return ldexp(p, (int)n);
}

// 2^a for -1/4 <= a <= 0: Taylor to a^10, whose rest is below (ln 2 / 4)^11 / 11! = 2^-53.
__device__ __forceinline__ double exp2_small(double a)
{
    double p = 7.0549116208011233299e-09;
    p = fma(p, a, 1.0178086009239699728e-07);
    p = fma(p, a, 1.3215486790144309488e-06);
    p = fma(p, a, 1.5252733804059840280e-05);
    p = fma(p, a, 1.5403530393381609954e-04);
    p = fma(p, a, 1.3333558146428443423e-03);
    p = fma(p, a, 9.6181291076284771620e-03);
    p = fma(p, a, 5.5504108664821579953e-02);
    p = fma(p, a, 2.4022650695910071233e-01);
    p = fma(p, a, 6.9314718055994530942e-01);
    return fma(p, a, 1.0);
}

__device__ __forceinline__ double weight(float x, float m, double c)
{
    return exp2_neg(((double)x - (double)m) * c);
}

// Four at once: each constant is fetched once for all of them.
__device__ __forceinline__ void exp2_neg4(const double (&a)[4], double (&w)[4])
{
    constexpr double C[14] = {1.3691488853904128881e-12, 2.5678435993488205142e-11, 4.4455382718708114976e-10,
                              7.0549116208011233299e-09, 1.0178086009239699728e-07, 1.3215486790144309488e-06,
                              1.5252733804059840280e-05, 1.5403530393381609954e-04, 1.3333558146428443423e-03,
                              9.6181291076284771620e-03, 5.5504108664821579953e-02, 2.4022650695910071233e-01,
                              6.9314718055994530942e-01, 1.0};
    double n[4], r[4];
    unroll<0, 4>([&](auto k) SV_INLINE {
        const double b = fmax(a[k], -1100.0);
        n[k] = rint(b);
        r[k] = b - n[k];
        w[k] = C[0];
    });
    unroll<1, 14>([&](auto i) SV_INLINE {
        unroll<0, 4>([&](auto k) SV_INLINE { w[k] = fma(w[k], r[k], C[i]); });
    });
    unroll<0, 4>([&](auto k) SV_INLINE { w[k] = ldexp(w[k], (int)n[k]); });
}

__device__ __forceinline__ void weight4(const float (&x)[4], float m, double c, double (&w)[4])
{
    double a[4];
    unroll<0, 4>([&](auto k) SV_INLINE { a[k] = ((double)x[k] - (double)m) * c; });
    exp2_neg4(a, w);
}

struct Params {
    double c;       // log2(e) / T
    double p, m;
    int k;          // 1..V
    bool ok;
};

// One row's or sequence's parameters: absent arrays cut nothing.  T = 0 is the first id of the
// order, which is k = 1 at any temperature.
__device__ __forceinline__ Params load_params(const FilterPtrs &f, int i, int V)
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
template <typename T> __device__ __forceinline__ T block_sum(T v, T *lds)
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

__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t *lds)
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

__device__ __forceinline__ bool kept(uint32_t key, int id, const RowCut &r)
{
    return key > r.cut || (key == r.cut && id <= r.tie);
}

// The row's cut by bisection on the order keys: every step is one pass over the row that counts
// or sums what lies above a key.  Exact for any row; 32 passes per active cut.
template <int DT>
__device__ __forceinline__ RowCut cut_by_bisection(const char *row, int V, const Params &q, RedLds &lds)
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
    r.kept = V;
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

// ------------------------------------------------------------------ reading a row
//
// Group g of a row is its ids g * E .. g * E + E - 1, one 16-byte vector.  Rows start at any
// element (an odd vocabulary, a stride), and the memory pipe takes 16-byte loads at any address,
// so the groups count from the row's first id whatever its alignment; only the last, partial
// group is read by elements.

typedef unsigned int u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

template <int DT> struct Groups {
    static constexpr int E = Elt<DT>::EPV;
    static constexpr uint32_t EMPTY = DT == 1 ? 0xff80ff80u : 0xff800000u;   // -inf
    const char *row;
    int V, whole, per_wave;    // whole groups; units of 64 groups that each wave takes in a draw

    __device__ __forceinline__ Groups(const char *r, int v) : row(r), V(v), whole(v / E)
    {
        per_wave = ((v + E - 1) / E + FWAVES * 64 - 1) / (FWAVES * 64);
    }
    __device__ __forceinline__ int group_of(int wave, int unit, int lane) const
    {
        return (wave * per_wave + unit) * 64 + lane;
    }
    __device__ __forceinline__ uint4 load_whole(int g) const
    {
        const u32x4_any v = *reinterpret_cast<const u32x4_any *>(row + (size_t)g * 16);
        return make_uint4(v.x, v.y, v.z, v.w);
    }
    // past the caches, for what is read once
    __device__ __forceinline__ uint4 load_once(int g) const
    {
        const u32x4_any v =
            __builtin_nontemporal_load(reinterpret_cast<const u32x4_any *>(row + (size_t)g * 16));
        return make_uint4(v.x, v.y, v.z, v.w);
    }
    // the last, partial group; -inf where it has no id
    __device__ __forceinline__ uint4 load_partial() const
    {
        uint32_t w0 = EMPTY, w1 = EMPTY, w2 = EMPTY, w3 = EMPTY;
#pragma nounroll
        for (int id = V - 1; id >= whole * E; --id) {
            if constexpr (DT == 1) {
                w3 = __builtin_amdgcn_alignbit(w3, w2, 16);
                w2 = __builtin_amdgcn_alignbit(w2, w1, 16);
                w1 = __builtin_amdgcn_alignbit(w1, w0, 16);
                w0 = w0 << 16 | reinterpret_cast<const uint16_t *>(row)[id];
            } else {
                w3 = w2;
                w2 = w1;
                w1 = w0;
                w0 = reinterpret_cast<const uint32_t *>(row)[id];
            }
        }
        return make_uint4(w0, w1, w2, w3);
    }
    // the group's logits; -inf where it has no id
    __device__ __forceinline__ uint4 load(int g) const
    {
        uint4 v = make_uint4(EMPTY, EMPTY, EMPTY, EMPTY);
        if (g < whole)
            v = load_whole(g);
        else if (g == whole && whole * E < V)
            v = load_partial();
        return v;
    }
};

__device__ __forceinline__ uint32_t vec_word(const uint4 &v, int i)
{
    return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}

// One of N vectors, the same in all lanes.
template <int N> __device__ __forceinline__ uint4 choose(const uint4 (&v)[N], int i)
{
    uint4 x = v[0];
    unroll<1, N>([&](auto j) SV_INLINE {
        if (j == i) {
            x = v[j];
            // keeps the choice a branch and four moves: merged, it would be an indexed read of an
            // array, which lives in memory
            asm volatile("" : "+v"(x.x), "+v"(x.y), "+v"(x.z), "+v"(x.w));
        }
    });
    return x;
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
constexpr int HBINS = 2 * HMAG;            // bin = sign * HMAG + magnitude - HLO: neighbouring
                                           // magnitudes lie in neighbouring LDS banks
constexpr int HX = 64;                     // values outside the window kept apart

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t as_u32(u16x2 v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ u16x2 as_u16x2(uint32_t v) { return __builtin_bit_cast(u16x2, v); }

// Two patterns less HLO; a half is inside the window exactly when its bits 12..14 are 0.
__device__ __forceinline__ uint32_t window_words(uint32_t w)
{
    const u16x2 lo = {(unsigned short)HLO, (unsigned short)HLO};
    return as_u32(as_u16x2(w) - lo);
}
// 4 * bin of both halves: magnitude in bits 2..13, sign in bit 14
__device__ __forceinline__ uint32_t bin_offsets(uint32_t t)
{
    const u16x2 two = {2, 2};
    return as_u32(as_u16x2(t) << two) | (t >> 1 & 0x40004000u);
}

__device__ __forceinline__ float pattern_value(uint32_t p) { return __uint_as_float(p << 16); }

// What masks write: values <= -2^8 and -inf.  As patterns less that of -2^8 they are the numbers up
// to MASK_INF, largest value first; every other pattern gives a larger one.
constexpr uint32_t MASK_TOP = 0xc380u, MASK_INF = 0xff80u - MASK_TOP;

__device__ __forceinline__ uint32_t mask_words(uint32_t w)
{
    const u16x2 top = {(unsigned short)MASK_TOP, (unsigned short)MASK_TOP};
    return as_u32(as_u16x2(w) - top);
}
// Not 0 where a half of window word t lies outside the window and, by mask word m, is not masked.
__device__ __forceinline__ uint32_t rare_words(uint32_t t, uint32_t m)
{
    const u16x2 inf = {(unsigned short)MASK_INF, (unsigned short)MASK_INF};
    return as_u32(__builtin_elementwise_min(__builtin_elementwise_sub_sat(as_u16x2(m), inf),
                                            as_u16x2(t & 0x70007000u)));
}
__device__ __forceinline__ uint32_t bin_pattern(int bin)
{
    return HLO + (uint32_t)(bin & (HMAG - 1)) + (bin >= HMAG ? 0x8000u : 0u);
}

// The order of a row's values as rows of four positions to a thread, largest first: row 0 the
// values above the window, then PR rows of positive bins, the values around zero, PR rows of
// negative bins.  Rows 0 and PR + 1 have one position to a lane of wave 0.
constexpr int order_rows(int wgt) { return 2 + 2 * (HMAG / (4 * wgt)); }

struct CutLds {
    uint32_t count[64];            // ids per order row and wave
    float first[64];               // the first value there
    double sum[64];                // kept weight there, after top-k
    float xval[2][64];             // the values kept apart, above the window and around zero
    uint32_t xcnt[2][64];
    uint32_t xlist[HX];            // patterns outside the window as they were met
    uint32_t nx, zeros, low, bad;  // how many; zeros; largest order key <= -2^8; NaN or +inf met
    int last[3];                   // last place that top-k, top-p, min-p leave something of
    uint32_t rth[2][FWAVES], top[2][FWAVES];  // per wave: a value that enough of its ids reach; its largest
    RowCut cut;
};

__device__ __forceinline__ void cut_lds_clear(CutLds &c)
{
    if (threadIdx.x == 0) {
        c.nx = c.zeros = c.low = c.bad = 0;
        c.last[0] = c.last[1] = c.last[2] = -1;
    }
}

__device__ __forceinline__ void count_outside(uint32_t p, CutLds &c)
{
    const uint32_t a = p & 0x7fffu;
    if (a == 0) {
        atomicAdd(&c.zeros, 1u);
    } else if (a >= 0x7f80u) {
        if (p != 0xff80u)
            atomicOr(&c.bad, 1u);
    } else {
        const uint32_t i = atomicAdd(&c.nx, 1u);
        if (i < HX)
            c.xlist[i] = p;
    }
}

__device__ __forceinline__ void bump(uint32_t *hist, uint32_t off)
{
    atomicAdd(reinterpret_cast<uint32_t *>(reinterpret_cast<char *>(hist) + off), 1u);
}

// Counts eight patterns.  The common case, all lanes inside the window, takes seven VALU
// instructions for two patterns and one LDS add for each.  Masked rows have -inf or low values
// anywhere, so these cost little more: left out of the adds, with the largest kept in `low`, the
// lane's least mask words.  (An LDS maximum for each of them took 500 us for a row of 152064 of
// which 70% had the type's lowest value.)
__device__ __forceinline__ void count_vec(const uint4 &v, uint32_t *hist, CutLds &c, uint32_t &low)
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
        return;
    }
    uint32_t rare = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t b = bin_offsets(t[i]), m = mask_words(vec_word(v, i));
        if ((t[i] & 0x7000u) == 0)
            bump(hist, b & 0xffffu);
        if ((t[i] & 0x70000000u) == 0)
            bump(hist, b >> 16);
        low = as_u32(__builtin_elementwise_min(as_u16x2(low), as_u16x2(m)));
        rare |= rare_words(t[i], m);
    }
    if (__ballot(rare != 0) != 0) {
        uint32_t w0 = v.x, w1 = v.y, w2 = v.z, w3 = v.w;
#pragma nounroll
        for (int i = 0; i < 8; ++i) {
            if (rare_words(window_words(w0), mask_words(w0)) & 0xffffu)
                count_outside(w0 & 0xffffu, c);
            w0 = __builtin_amdgcn_alignbit(w1, w0, 16);
            w1 = __builtin_amdgcn_alignbit(w2, w1, 16);
            w2 = __builtin_amdgcn_alignbit(w3, w2, 16);
            w3 >>= 16;
        }
    }
}

constexpr uint32_t NO_LOW = 0xffffffffu;

// The wave's largest value <= -2^8, if it met one.
__device__ __forceinline__ void note_low(uint32_t low, CutLds &c)
{
    int m = (int)min(low & 0xffffu, low >> 16);
    if (__ballot(m < (int)MASK_INF) == 0)
        return;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1)
        m = min(m, __shfl_xor(m, o));
    if ((threadIdx.x & 63) == 0)
        atomicMax(&c.low, order_key(pattern_value(MASK_TOP + (uint32_t)m)));
}

__device__ __forceinline__ uint32_t wave_scan_u32(uint32_t x)
{
    int v = (int)x;
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);  // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);  // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);  // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31
    return (uint32_t)v;
}

// What need not be counted.  With top-k, an id cannot matter once k others are known to be above
// it; with min-p and neither of the others, once it lies too far below a maximum.  Each wave notes
// in LDS the r-th largest of its lanes' maxima so far, r = ceil(k / waves): the waves' least is a
// value that at least k ids reach.  Groups below it cost two instructions for a pair of logits, in
// place of two LDS adds, and after the first part of a row nearly all are.  Only floors above zero
// are used, where patterns compare as signed integers.  The waves wait for each other's notes, so
// that what is counted and listed, and with it the grouping of every sum, is the same in each run.
typedef short s16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ s16x2 as_s16x2(uint32_t v) { return __builtin_bit_cast(s16x2, v); }
__device__ __forceinline__ uint32_t max_i16(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(as_s16x2(a), as_s16x2(b)));
}
__device__ __forceinline__ uint32_t max_u16(uint32_t a, uint32_t b)
{
    return as_u32(__builtin_elementwise_max(as_u16x2(a), as_u16x2(b)));
}
__device__ __forceinline__ uint32_t group_max(const uint4 &v)
{
    return max_i16(max_i16(v.x, v.y), max_i16(v.z, v.w));
}

struct Floor {
    bool by_k, by_m;
    int r;
    float drop;              // T ln m, a little lower
    uint32_t top = 0x80008000u, most = 0;    // the lane's largest: signed, and as unsigned patterns
    uint32_t below = 0;      // the largest pattern, twice, that need not be counted; 0: none

    __device__ __forceinline__ Floor(const Params &q, int V, int waves)
    {
        by_k = q.k < V && q.k <= 64 * waves;
        by_m = q.p >= 1.0 && q.m > 0.0 && (q.k >= V || by_k);
        r = (q.k + waves - 1) / waves;
        drop = by_m ? (float)(log2(q.m) / q.c * 1.00001) - 1e-30f : 0.0f;
    }
    __device__ __forceinline__ bool active() const { return by_k || by_m; }
    __device__ __forceinline__ void see(const uint4 &v)
    {
        top = max_i16(top, group_max(v));
        most = max_u16(most, max_u16(max_u16(v.x, v.y), max_u16(v.z, v.w)));
    }
    // Notes the wave's bounds, and takes the floor from all waves' notes, in steps 0, 3, 15 and 63 of
    // the row: more of them raise it little and make the waves wait (in steps 0, 1, 3, 7, ... a verify
    // B=64 K=5 V=32000 in float32 takes 68.4 us, so 65.3; B=17 K=3 V=50257 in bfloat16 44.8 and 43.5).
    // All waves of the workgroup come here in every step.  Two sets of notes in turn: who writes one
    // again has waited once more since it was read.
    template <int NW> __device__ __forceinline__ void exchange(CutLds &c, int step)
    {
        if ((step & (step + 1)) != 0 || (__popc(step) & 1) != 0)
            return;
        const int turn = __popc(step) / 2;
        const int wv = threadIdx.x >> 6;
        const int a = (int)(short)(top & 0xffffu), b = (int)(short)(top >> 16), best = max(max(a, b), 0);
        int t = 0, mx = 0;
#pragma unroll
        for (int bit = 14; bit >= 0; --bit) {
            const int u = t | 1 << bit, w = mx | 1 << bit;
            if (__popcll(__ballot(best >= u)) >= r)
                t = u;
            if (__ballot(best >= w) != 0)
                mx = w;
        }
        uint32_t *rth = c.rth[turn & 1], *tops = c.top[turn & 1];
        if ((threadIdx.x & 63) == 0) {
            rth[wv] = (uint32_t)t;
            tops[wv] = (uint32_t)mx;
        }
        __syncthreads();
        const int lane = threadIdx.x & (NW - 1);
        int k = (int)rth[lane], m = (int)tops[lane];
        k = min(k, lane_xch<0>(k));
        m = max(m, lane_xch<0>(m));
        k = min(k, lane_xch<1>(k));
        m = max(m, lane_xch<1>(m));
        k = min(k, lane_xch<2>(k));
        m = max(m, lane_xch<2>(m));
        if (NW > 8) {
            k = min(k, lane_xch<3>(k));
            m = max(m, lane_xch<3>(m));
        }
        static_assert(NW == 8 || NW == 16, "lanes exchanged over the waves' notes");
        uint32_t f = by_k ? (uint32_t)k : 0;
        if (by_m) {
            const float y = pattern_value((uint32_t)m) + drop;
            if (m < 0x7f80 && y > 0.0f)
                f = max(f, __float_as_uint(y) >> 16);
        }
        // NaN and +inf are counted, so that they are seen
        f = min(f, 0x7f80u);
        below = __builtin_amdgcn_readfirstlane(f > 1 ? (f - 1) * 0x10001u : 0);
    }
    __device__ __forceinline__ bool matters(const uint4 &v) const
    {
        return below == 0 || max_i16(group_max(v), below) != below;
    }
    // a NaN of negative sign lies below any floor
    __device__ __forceinline__ uint32_t bad() const
    {
        return (most & 0xffffu) > 0xff80u || most >> 16 > 0xff80u;
    }
};

// The values kept apart, in order, into xval and xcnt (wave 0).
__device__ __forceinline__ void order_outside(CutLds &c)
{
    const int lane = threadIdx.x & 63;
    c.xcnt[0][lane] = c.xcnt[1][lane] = 0;
    c.xval[0][lane] = c.xval[1][lane] = 0.0f;
    const int n = (int)min(c.nx, (uint32_t)HX - 1);
    if (n == 0) {
        if (lane == 0)
            c.xcnt[1][0] = c.zeros;
        return;
    }
    // lane n stands for the zeros; of equal values the first stands for all
    const float x = lane < n ? pattern_value(c.xlist[lane]) : 0.0f;
    const uint32_t mine = lane < n ? 1u : lane == n ? c.zeros : 0u;
    const bool high = x >= 256.0f;
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
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// The thread's four positions of an order row: counts, values and first bin (-1 outside the
// window; positive bins descend from it, negative ones ascend).
template <int WGT>
__device__ __forceinline__ void order_entry(int row, const uint32_t *hist, const CutLds &c, uint32_t (&n)[4],
                                   float (&x)[4], int &bin)
{
    constexpr int PR = HMAG / (4 * WGT);
    const int t = threadIdx.x;
    if (row == 0 || row == PR + 1) {
        const bool in = t < 64;
        n[0] = in ? c.xcnt[row != 0][t & 63] : 0u;
        x[0] = in ? c.xval[row != 0][t & 63] : 0.0f;
        n[1] = n[2] = n[3] = 0;
        x[1] = x[2] = x[3] = 0.0f;
        bin = -1;
        return;
    }
    const bool neg = row > PR + 1;
    const int at = 4 * ((neg ? row - PR - 2 : row - 1) * WGT + t);
    bin = neg ? HMAG + at : HMAG - 1 - at;
    const uint4 q = *reinterpret_cast<const uint4 *>(hist + (neg ? bin : bin - 3));
    n[0] = neg ? q.x : q.w;
    n[1] = neg ? q.y : q.z;
    n[2] = neg ? q.z : q.y;
    n[3] = neg ? q.w : q.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        x[i] = pattern_value(bin_pattern(neg ? bin + i : bin - i));
}

// The cut from the counts, by a workgroup of WGT threads; on return c.cut holds it.  Top-k, top-p
// and min-p each leave a prefix of the order, so the cut lies in the first of the three places
// (order row, thread) where theirs end, and there position by position.  With `table`,
// table[bin] receives the weight of every bin that occurs and is kept, and 0 of every bin that
// occurs and is not.  `whole`: every id was counted, not just those that matter.
template <int WGT>
__device__ __forceinline__ void cut_from_counts(const uint32_t *hist, CutLds &c, const Params &q, int V,
                                                bool whole, double *table)
{
    constexpr int NW = WGT / 64, R = order_rows(WGT);
    static_assert(R * NW <= 64, "a lane for every order row and wave");
    const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
    __syncthreads();
    if (wv == 0)
        order_outside(c);
    // wave 0 alone reads what it has just written there
    uint32_t cnt[R], before[R];
    unroll<0, R>([&](auto r) SV_INLINE {
        uint32_t n[4];
        float x[4];
        int bin;
        order_entry<WGT>(r, hist, c, n, x, bin);
        cnt[r] = n[0] + n[1] + n[2] + n[3];
        const unsigned long long has = __ballot(cnt[r] != 0);
        uint32_t inc = 0;
        if (has) {
            inc = wave_scan_u32(cnt[r]);
            if (lane == __ffsll(has) - 1)
                c.first[r * NW + wv] = n[0] ? x[0] : n[1] ? x[1] : n[2] ? x[2] : x[3];
        }
        before[r] = inc - cnt[r];
        if (lane == 63)
            c.count[r * NW + wv] = inc;
    });
    __syncthreads();
    const uint32_t mine = lane < R * NW ? c.count[lane] : 0u;
    const uint32_t inc = wave_scan_u32(mine);
    const uint32_t total = (uint32_t)lane_value((int)inc, 63);
    const unsigned long long some = __ballot(mine != 0);
    const float M = some ? c.first[__ffsll(some) - 1] : 0.0f;
    unroll<0, R>([&](auto r) SV_INLINE {
        before[r] += (uint32_t)lane_value((int)(inc - mine), r * NW + __builtin_amdgcn_readfirstlane(wv));
    });
    RowCut cut;
    cut.z = 0.0;
    cut.c = q.c;
    cut.max = M;
    cut.cut = KEY_NEG_INF;
    cut.tie = V;
    cut.state = CUT_READY;
    cut.kept = V;
    if (!q.ok || c.bad || (total == 0 && c.low == 0)) {
        cut.state = CUT_NONE;
    } else if (c.nx >= HX || total == 0) {
        cut.state = CUT_EXACT;
    } else if (c.low) {
        // the low values count if one of them could be kept with a weight that matters; with p = 1
        // none is that min-p leaves out, however few were counted above its floor
        const double w = weight(key_value(c.low), M, q.c);
        const bool left_out = q.p >= 1.0 && w < q.m;
        if (w > 0.0 && !left_out &&
            (w >= 0x1p-80 || (q.k < V && q.k > (int)total) || (q.m > 0.0 && w >= q.m)))
            cut.state = CUT_EXACT;
    }
    if (cut.state != CUT_READY) {
        if (t == 0)
            c.cut = cut;
        __syncthreads();
        return;
    }
    const uint32_t k = min((uint32_t)q.k, total);
    double sum[R];
    uint32_t passes = 0;       // bit r: min-p leaves something of the thread's positions in row r
    unroll<0, R>([&](auto r) SV_INLINE {
        sum[r] = 0.0;
        const bool in = cnt[r] != 0 && before[r] < k;
        if (__ballot(cnt[r] != 0) == 0) {
            if (lane == 63)
                c.sum[r * NW + wv] = 0.0;
            return;
        }
        if (__ballot(in) != 0) {
            uint32_t n[4];
            float x[4];
            int bin;
            order_entry<WGT>(r, hist, c, n, x, bin);
            uint32_t b = before[r];
            double w[4];
            weight4(x, M, q.c, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t left = b >= k ? 0u : min(n[i], k - b);
                b += n[i];
                w[i] = left ? w[i] : 0.0;      // what does not occur may lie above M
                sum[r] += (double)left * w[i];
                passes |= (uint32_t)(left && w[i] >= q.m) << r;
            }
            if (table && bin >= 0 && cnt[r] != 0) {
                const bool neg = bin >= HMAG;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    table[neg ? bin + i : bin - i] = w[i];
            }
        } else if (table && cnt[r] != 0) {
            // occurs, but past the first k
            uint32_t n[4];
            float x[4];
            int bin;
            order_entry<WGT>(r, hist, c, n, x, bin);
            if (bin >= 0)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    table[bin >= HMAG ? bin + i : bin - i] = 0.0;
        }
        const double s = wave_incl_scan(sum[r]);
        if (lane == 63)
            c.sum[r * NW + wv] = s;
        sum[r] = wave_excl_from_incl(s);       // from here on: what lies before the thread
    });
    __syncthreads();
    const double wmine = lane < R * NW ? c.sum[lane] : 0.0, winc = wave_incl_scan(wmine);
    const double zk = lane_value(winc, 63), wexc = wave_excl_from_incl(winc);
    const double goal = q.p < 1.0 ? q.p * zk : INFINITY;
    int last[3] = {-1, -1, -1};
    unroll<0, R>([&](auto r) SV_INLINE {
        sum[r] += lane_value(wexc, r * NW + __builtin_amdgcn_readfirstlane(wv));
        const bool in = cnt[r] != 0 && before[r] < k;
        const unsigned long long a = __ballot(in);
        const unsigned long long b = __ballot(in && (sum[r] < goal || before[r] == 0));
        const unsigned long long m = __ballot(passes >> r & 1);
        if (a)
            last[0] = r * WGT + wv * 64 + 63 - __clzll(a);
        if (b)
            last[1] = r * WGT + wv * 64 + 63 - __clzll(b);
        if (m)
            last[2] = r * WGT + wv * 64 + 63 - __clzll(m);
    });
    const int mylast = lane == 0 ? last[0] : lane == 1 ? last[1] : last[2];
    if (lane < 3 && mylast >= 0)
        atomicMax(&c.last[lane], mylast);
    __syncthreads();
    const int owner = min(c.last[0], min(c.last[1], c.last[2]));
    const bool all = whole && q.p >= 1.0 && k == total && q.m <= 0.0;
    if (all) {
        if (t == 0) {
            cut.z = zk;
            c.cut = cut;
        }
    } else {
        // the owner's row, the same in all threads
        const int at = __builtin_amdgcn_readfirstlane(owner / WGT);
        uint32_t b0 = 0;
        double run = 0.0;
        unroll<0, R>([&](auto r) SV_INLINE {
            b0 = r == at ? before[r] : b0;
            run = r == at ? sum[r] : run;
            // the bins past the owner's
            if (table && cnt[r] != 0 && r * WGT + t > owner && r != 0 && r != R / 2) {
                constexpr bool neg = r > R / 2;
                const int p = 4 * ((neg ? r - R / 2 - 1 : r - 1) * WGT + t);
                double2 *q = reinterpret_cast<double2 *>(table + (neg ? HMAG + p : HMAG - 4 - p));
                q[0] = q[1] = make_double2(0.0, 0.0);
            }
        });
        if (at * WGT + t == owner) {
            uint32_t n[4];
            float x[4];
            int bin, keep_to = -1;         // the last of the four positions kept
            order_entry<WGT>(at, hist, c, n, x, bin);
            uint32_t b = b0;
            bool go = true;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t left = b >= k ? 0u : min(n[i], k - b);
                const double w = left ? weight(x[i], M, q.c) : 0.0;
                if (go && left) {
                    go = (run < goal || b == 0) && w >= q.m;
                    if (go) {
                        uint32_t keep = left;
                        if (q.p < 1.0) {
                            const double f = ceil((goal - run) / w);
                            keep = f < 1.0 ? 1u : f > (double)left ? left : (uint32_t)f;
                        }
                        keep_to = i;
                        cut.cut = order_key(x[i]);
                        cut.z = run + (double)keep * w;
                        cut.state = keep < n[i] ? CUT_TIES : CUT_READY;
                        cut.tie = keep < n[i] ? (int)keep : V;
                        cut.kept = b + keep;
                    }
                }
                b += n[i];
                run += (double)left * w;
            }
            c.cut = cut;
            if (table && bin >= 0)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i > keep_to)
                        table[bin >= HMAG ? bin + i : bin - i] = 0.0;
        }
    }
    __syncthreads();
}

// Counts a row straight from memory, COUNT_LOADS vectors of a thread in flight; the other waves of
// the compute unit count meanwhile.
constexpr int COUNT_LOADS = 4;

template <int WGT>
__device__ __forceinline__ void count_row(const Groups<1> &gr, Floor &fl, uint32_t *hist, CutLds &c)
{
    constexpr int U = COUNT_LOADS, NW = WGT / 64;
    const int t = threadIdx.x;
    uint32_t low = NO_LOW;
#pragma nounroll
    for (int i = 0; i * U * WGT < gr.whole; ++i) {
        const int g = i * U * WGT + t;
        uint4 v[U];
        const bool full = (i + 1) * U * WGT <= gr.whole;
        // threads past the end read the last group again and drop it
        unroll<0, U>([&](auto k) SV_INLINE { v[k] = gr.load_once(min(g + k * WGT, gr.whole - 1)); });
        if (!full)
            unroll<0, U>([&](auto k) SV_INLINE {
                if (g + k * WGT >= gr.whole)
                    v[k] = make_uint4(gr.EMPTY, gr.EMPTY, gr.EMPTY, gr.EMPTY);
            });
        if (fl.active()) {
            unroll<0, U>([&](auto k) SV_INLINE { fl.see(v[k]); });
            fl.template exchange<NW>(c, i);
        }
        if (full && fl.below == 0) {
            unroll<0, U>([&](auto k) SV_INLINE { count_vec(v[k], hist, c, low); });
        } else {
            unroll<0, U>([&](auto k) SV_INLINE {
                if (g + k * WGT < gr.whole && fl.matters(v[k]))
                    count_vec(v[k], hist, c, low);
            });
        }
    }
    if (t == 0 && gr.whole * 8 < gr.V) {
        const uint4 x = gr.load_partial();
        fl.see(x);
        count_vec(x, hist, c, low);
    }
    note_low(low, c);
    if (fl.active() && fl.bad())
        atomicOr(&c.bad, 1u);
}

template <int WGT> __device__ __forceinline__ void clear_hist(uint32_t *hist)
{
    for (int i = threadIdx.x; i < HBINS / 4; i += WGT)
        reinterpret_cast<uint4 *>(hist)[i] = make_uint4(0, 0, 0, 0);
}

constexpr int RWG = 512;   // threads per row of a bfloat16 verify: four workgroups to a compute unit

// The RowCut of every target and draft row of a bfloat16 verify.  Four workgroups of 35 KB to a
// compute unit, so that one counts while another is at its cut's barriers: 4352 rows of 128256
// (1.12 GB) take 170 us, 6.6 TB/s, where a bare streaming read of the same layout takes 161-164.
// Counting is seven VALU instructions and two LDS adds for two logits: in those 170 us a SIMD issues
// 62 thousand VALU instructions (246 thousand clocks) and a compute unit's LDS works for 113
// thousand, so that the reads hide both, but not by much.
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
    Floor fl(q, V, RWG / 64);
    count_row<RWG>(Groups<1>(row, V), fl, hist, c);
    cut_from_counts<RWG>(hist, c, q, V, !fl.active(), nullptr);
    if (threadIdx.x == 0)
        cuts[n] = c.cut;
}

// ------------------------------------------------------------------ the inverse-CDF draw
//
// Each of a workgroup's waves takes a contiguous range of a row's groups, 64 at a time (a unit).
// The waves' kept weights decide which of them holds the id whose cumulative weight passes
// u * total, and that wave goes over its units again, in order, to the unit, the lane and the id.
// All sums have a fixed order.

constexpr int LIST = 256;  // groups that matter in a wave's range, if they are so few

struct DrawLds {
    double batch[FWAVES][64];
    double wave[FWAVES];
    double total;              // the row's
    int ties[2][FWAVES], tie_id[2];
    uint16_t list[FWAVES][LIST];
    int id;
};

// A wave's groups, in order and 64 to a unit: all of its range, or a list of those that matter.
template <int DT> struct Units {
    const Groups<DT> &gr;
    const uint16_t *list;
    int n;                 // length of the list, -1 for the whole range

    __device__ __forceinline__ int first() const
    {
        return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * gr.per_wave * 64;
    }
    // units that hold a group of the row
    __device__ __forceinline__ int count() const
    {
        const int groups = (gr.V + gr.E - 1) / gr.E;
        return n < 0 ? max(0, min(gr.per_wave, (groups - first() + 63) / 64)) : (n + 63) / 64;
    }
    // the lane's group of unit i; past the row or the list's end, one that holds() is false for
    __device__ __forceinline__ int group(int i) const
    {
        const int at = i * 64 + (threadIdx.x & 63);
        return n < 0 ? first() + at : first() + list[at < n ? at : i * 64];
    }
    __device__ __forceinline__ bool holds(int i) const
    {
        return n < 0 || i * 64 + (int)(threadIdx.x & 63) < n;
    }
};

// A wave's units are read four at a time (a batch), all four loads in flight.  A wave notes in
// a bit per batch where there was something for it, and later passes read only those.
constexpr int BATCH = 4;
static_assert((MAX_VOCAB / 4 + FWAVES * 64 - 1) / (FWAVES * 64) <= 64 * BATCH, "a bit for every batch");

template <int DT>
__device__ __forceinline__ void load_batch(const Units<DT> &un, int i0, uint4 (&v)[BATCH])
{
    const Groups<DT> &gr = un.gr;
    const int units = un.count(), g0 = un.first() + i0 * 64, lane = threadIdx.x & 63;
    if (un.n < 0 && i0 + BATCH <= units && g0 + BATCH * 64 <= gr.whole) {
        unroll<0, BATCH>([&](auto j) SV_INLINE { v[j] = gr.load_whole(g0 + j * 64 + lane); });
        return;
    }
    unroll<0, BATCH>([&](auto j) SV_INLINE {
        v[j] = make_uint4(gr.EMPTY, gr.EMPTY, gr.EMPTY, gr.EMPTY);
        if (i0 + j < units) {
            const int g = un.group(i0 + j);
            if (g < gr.whole)
                v[j] = gr.load_whole(g);
        }
    });
    if (gr.whole * gr.E < gr.V) {
        const uint4 last = gr.load_partial();
        unroll<0, BATCH>([&](auto j) SV_INLINE {
            if (i0 + j < units && un.group(i0 + j) == gr.whole)
                v[j] = last;
        });
    }
}

template <int DT> __device__ __forceinline__ uint64_t all_batches(const Units<DT> &un)
{
    const int n = (un.count() + BATCH - 1) / BATCH;
    return n >= 64 ? ~0ull : (1ull << n) - 1;
}

// Adds the lanes' groups `at` for which m holds to a wave's list, in order, of which n are listed
// already; past LIST they are only counted.
__device__ __forceinline__ void list_groups(uint16_t *list, int &n, bool m, int at)
{
    const unsigned long long who = __ballot(m);
    if (who) {
        const int i = n + (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32),
                                                         __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0));
        n += __popcll(who);
        if (m && i < LIST)
            list[i] = (uint16_t)at;
    }
}

// The units of batch i0 that may() something in, as a mask, and their aux() groups.
template <int DT, typename A, typename W>
__device__ __forceinline__ uint32_t look(const Units<DT> &un, int i0, const uint4 (&v)[BATCH],
                                         uint4 (&x)[BATCH], A may, const W &law)
{
    uint32_t mask = 0;
    const int units = un.count();
    unroll<0, BATCH>([&](auto j) SV_INLINE {
        if (i0 + j < units && __ballot(may(v[j])) != 0) {
            mask |= 1u << j;
            x[j] = law.aux(un.group(i0 + j));
        }
    });
    return __builtin_amdgcn_readfirstlane(mask);
}

// The draw.  Every wave sums its batches of units; the wave that holds the id then looks again at
// the batch that holds it.  law.sum(g, vec, law.aux(g)) is the weight of a group, law.one(logit, id)
// that of one id.  Returns the id in every thread, -1 if all weights are 0.
template <int DT, typename A, typename W>
__device__ __forceinline__ int draw_row(const Units<DT> &un, A may, double u, DrawLds &lds,
                                        const W &law)
{
    constexpr int E = Elt<DT>::EPV;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, units = un.count();
    if (threadIdx.x == 0)
        lds.id = -1;
    uint64_t with = 0;             // batches with some weight
    double all = 0.0;
    uint4 nx[BATCH];
    if (W::AHEAD)
        load_batch(un, 0, nx);
#pragma nounroll
    for (int i0 = 0; i0 < units; i0 += BATCH) {
        uint4 v[BATCH], x[BATCH];
        if constexpr (W::AHEAD) {
            unroll<0, BATCH>([&](auto j) SV_INLINE { v[j] = nx[j]; });
            if (i0 + BATCH < units)
                load_batch(un, i0 + BATCH, nx);
        } else {
            load_batch(un, i0, v);
        }
        const uint32_t mask = look(un, i0, v, x, may, law);
        if (!mask)
            continue;
        double mine = 0.0;
        unroll<0, BATCH>([&](auto j) SV_INLINE {
            if (mask >> j & 1) {
                const double s = law.sum(un.group(i0 + j), v[j], x[j]);
                mine += un.holds(i0 + j) ? s : 0.0;
            }
        });
        const double s = lane_value(wave_incl_scan(mine), 63);
        if (s > 0.0) {
            with |= 1ull << i0 / BATCH;
            all += s;
            if (lane == 0)
                lds.batch[wv][i0 / BATCH] = s;
        }
    }
    if (lane == 0)
        lds.wave[wv] = all;
    __syncthreads();
    // lane w: wave w's sum
    const double ws = lane < FWAVES ? lds.wave[lane] : 0.0, wi = wave_incl_scan(ws);
    double goal = u * lane_value(wi, 63);
    if (threadIdx.x == 0)
        lds.total = lane_value(wi, 63);
    const unsigned long long pos = __ballot(ws > 0.0), over = __ballot(ws > 0.0 && wi > goal);
    const int pick = over ? __ffsll(over) - 1 : pos ? 63 - __clzll(pos) : -1;
    if (__builtin_amdgcn_readfirstlane(wv) == pick) {
        // where rounding leaves no batch, unit, lane or id above the goal: the last of positive weight
        if (!over)
            goal = INFINITY;
        double base = lane_value(wave_excl_from_incl(wi), pick), before = base;
        bool found = false;
        int at = 0;
#pragma nounroll
        for (; with && !found; with &= with - 1) {
            at = __builtin_ctzll(with);
            const double s = lds.batch[wv][at];
            before = base;
            base += s;
            found = base > goal;
        }
        if (!found)
            goal = INFINITY;
        base = before;
        uint4 v[BATCH], x[BATCH], uv = make_uint4(0, 0, 0, 0);
        load_batch(un, at * BATCH, v);
        uint32_t mask = look(un, at * BATCH, v, x, may, law);
        double us = 0.0;           // the unit's: lane sums, groups, what lies before
        int ug = 0;
        found = false;
#pragma nounroll
        for (; mask && !found; mask &= mask - 1) {
            const int j = __builtin_ctz(mask), i = at * BATCH + j, g = un.group(i);
            const uint4 w = choose(v, j);
            const double s0 = law.sum(g, w, choose(x, j)), s = un.holds(i) ? s0 : 0.0;
            const double sum = lane_value(wave_incl_scan(s), 63);
            if (sum > 0.0) {
                us = s;
                ug = g;
                uv = w;
                before = base;
                base += sum;
                found = base > goal;
            }
        }
        if (!found)
            goal = INFINITY;
        const double inc = wave_incl_scan(us);
        const unsigned long long lpos = __ballot(us > 0.0);
        const unsigned long long lover = __ballot(us > 0.0 && before + inc > goal);
        const int l = lover ? __ffsll(lover) - 1 : 63 - __clzll(lpos);
        before += lane_value(wave_excl_from_incl(inc), l);
        // lane k: the group's k-th id
        const uint32_t w[4] = {(uint32_t)lane_value((int)uv.x, l), (uint32_t)lane_value((int)uv.y, l),
                               (uint32_t)lane_value((int)uv.z, l), (uint32_t)lane_value((int)uv.w, l)};
        const int k = lane % E, id = lane_value(ug, l) * E + k, word = DT == 1 ? k / 2 : k;
        const uint32_t b = word == 0 ? w[0] : word == 1 ? w[1] : word == 2 ? w[2] : w[3];
        const float y = DT == 1 ? pattern_value(k & 1 ? b >> 16 : b & 0xffffu) : __uint_as_float(b);
        const double p = lane < E && id < un.gr.V ? law.one(y, id) : 0.0, pi = wave_incl_scan(p);
        const unsigned long long ppos = __ballot(p > 0.0);
        const unsigned long long pover = __ballot(p > 0.0 && lover && before + pi > goal);
        if (lane == (pover ? __ffsll(pover) - 1 : 63 - __clzll(ppos)))
            lds.id = id;
    }
    __syncthreads();
    return lds.id;
}

// Bit k: the k-th logit of the group equals y.
template <int DT> __device__ __forceinline__ uint32_t equal_mask(const uint4 &v, float y)
{
    float x[Elt<DT>::EPV];
    Elt<DT>::unpack(v, x);
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < Elt<DT>::EPV; ++k)
        m |= (uint32_t)(x[k] == y) << k;
    return m;
}

// How many logits of the group equal y; bfloat16 two at a time, as patterns (the zeros without
// their sign).
template <int DT> __device__ __forceinline__ uint32_t equal_count(const uint4 &v, float y)
{
    if constexpr (DT == 1) {
        const uint32_t keep = y == 0.0f ? 0x7fff7fffu : 0xffffffffu;
        const uint32_t p = (__float_as_uint(y) >> 16) * 0x10001u & keep;
        const u16x2 one = {1, 1};
        u16x2 n = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            n += __builtin_elementwise_min(as_u16x2((vec_word(v, i) & keep) ^ p), one);
        return 8u - n.x - n.y;
    } else {
        return __popc(equal_mask<DT>(v, y));
    }
}

// Whether a group can hold a kept id.  bfloat16: for a cut above zero patterns compare as signed
// 16-bit integers, two at a time; else any group may.
template <int DT> struct MayKeep {
    uint32_t below;      // bfloat16: the largest pattern, twice, below the cut; 0: any group may
    float low;           // float32: the cut
    __device__ __forceinline__ explicit MayKeep(const RowCut &r)
    {
        low = key_value(r.cut);
        below = DT == 1 && low > 0.0f ? ((__float_as_uint(low) >> 16) - 1) * 0x10001u : 0;
    }
    __device__ __forceinline__ bool operator()(const uint4 &v) const
    {
        if constexpr (DT == 1)
            return below == 0 || max_i16(group_max(v), below) != below;
        else
            return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)),
                         fmaxf(__uint_as_float(v.z), __uint_as_float(v.w))) >= low;
    }
};

// Values that are the same in all lanes, kept in scalar registers: the laws' parameters would else
// take some 30 vector registers of a draw that has none to spare.
__device__ __forceinline__ double uniform(double x) { return lane_value(x, 0); }
__device__ __forceinline__ RowCut uniform(RowCut r)
{
    r.z = uniform(r.z);
    r.c = uniform(r.c);
    r.max = __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(r.max)));
    r.cut = (uint32_t)__builtin_amdgcn_readfirstlane((int)r.cut);
    r.tie = __builtin_amdgcn_readfirstlane(r.tie);
    return r;
}

// Finds, for up to two rows at once, the last kept id among those equal to a cut, the n-th of
// them: equals per batch and wave, then the unit, the lane and the id.  need: bit 0 p, bit 1 q,
// bit 2: list the groups of p (all of its range) that can hold a kept id.  Returns the list's
// length, -1 if it is too long or not asked for.
template <int DT>
__device__ __forceinline__ int find_ties(const Units<DT> &up, const Units<DT> &uq, int need, RowCut &rp,
                                         RowCut &rq, DrawLds &lds)
{
    const MayKeep<DT> may(rp);
    int listed = 0;
    constexpr int E = Elt<DT>::EPV;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int units = max(need & 5 ? up.count() : 0, need & 2 ? uq.count() : 0);
    const float yp = key_value(rp.cut), yq = key_value(rq.cut);
    uint32_t *batch = reinterpret_cast<uint32_t *>(lds.batch[wv]);
    int allp = 0, allq = 0;
    // a batch holds at most 2048 ids: two counts to a word
#pragma nounroll
    for (int i0 = 0; i0 < units; i0 += BATCH) {
        uint4 p[BATCH], q[BATCH];
        if (need & 5)
            load_batch(up, i0, p);
        if (need & 2)
            load_batch(uq, i0, q);
        uint32_t n = 0;
        if (need & 4)
            unroll<0, BATCH>([&](auto j) SV_INLINE {
                list_groups(lds.list[wv], listed, i0 + j < units && may(p[j]), (i0 + j) * 64 + lane);
            });
        if (need & 1)
            unroll<0, BATCH>([&](auto j) SV_INLINE {
                n += i0 + j < up.count() && up.holds(i0 + j) ? equal_count<DT>(p[j], yp) : 0u;
            });
        if (need & 2)
            unroll<0, BATCH>([&](auto j) SV_INLINE {
                n += (i0 + j < uq.count() && uq.holds(i0 + j) ? equal_count<DT>(q[j], yq) : 0u) << 16;
            });
        const uint32_t s = (uint32_t)lane_value((int)wave_scan_u32(n), 63);
        allp += (int)(s & 0xffffu);
        allq += (int)(s >> 16);
        if (lane == 0)
            batch[i0 / BATCH] = s;
    }
    if (lane == 0) {
        lds.ties[0][wv] = allp;
        lds.ties[1][wv] = allq;
    }
    if (threadIdx.x < 2)
        lds.tie_id[threadIdx.x] = 0x7fffffff;
    __syncthreads();
#pragma nounroll
    for (int side = 0; side < 2; ++side) {
        if (!(need >> side & 1))
            continue;
        const int n = side ? rq.tie : rp.tie;
        const int w = lane < FWAVES ? lds.ties[side][lane] : 0, wi = (int)wave_scan_u32((uint32_t)w);
        const int me = __builtin_amdgcn_readfirstlane(wv);
        int before = lane_value(wi - w, me);
        if (!(before < n && n <= lane_value(wi, me)))
            continue;
        int at = 0;
        for (;; ++at) {                        // ends: the wave's batches hold the n-th
            const int s = (int)(side ? batch[at] >> 16 : batch[at] & 0xffffu);
            if (before + s >= n)
                break;
            before += s;
        }
        const Units<DT> un{side ? uq.gr : up.gr, side ? uq.list : up.list, side ? uq.n : up.n};
        uint4 v[BATCH];
        load_batch(un, at * BATCH, v);
#pragma nounroll
        for (int j = 0; j < BATCH; ++j) {
            const int i = at * BATCH + j;
            if (i >= un.count())
                break;
            uint32_t m = un.holds(i) ? equal_mask<DT>(choose(v, j), side ? yq : yp) : 0u;
            const int c = __popc(m), inc = before + (int)wave_scan_u32((uint32_t)c), b = inc - c;
            if (b < n && n <= inc) {
                for (int skip = n - b - 1; skip > 0; --skip)
                    m &= m - 1;
                lds.tie_id[side] = un.group(i) * E + __ffs(m) - 1;
            }
            before = lane_value(inc, 63);
        }
    }
    __syncthreads();
    if (need & 1)
        rp.tie = lds.tie_id[0];
    if (need & 2)
        rq.tie = lds.tie_id[1];
    __syncthreads();
    return need & 4 && listed <= LIST ? __builtin_amdgcn_readfirstlane(listed) : -1;
}

// How many ids below x equal y.
template <int DT>
__device__ __forceinline__ int equals_below(const Groups<DT> &gr, int x, float y, RedLds &red)
{
    constexpr int E = Elt<DT>::EPV;
    const int last = x / E;
    int n = 0;
    for (int g0 = threadIdx.x; g0 <= last; g0 += 8 * FWG) {
        uint4 v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = gr.load(min(g0 + j * FWG, last));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int g = g0 + j * FWG;
            uint32_t m = equal_mask<DT>(v[j], y);
            if (g == last)
                m &= (1u << (x % E)) - 1;
            n += g <= last ? __popc(m) : 0;
        }
    }
    return block_sum(n, red.i);
}

// The logits of a group one after another: the first of w[], which moves on.
template <int DT> __device__ __forceinline__ float next_logit(uint32_t (&w)[4])
{
    float x;
    if constexpr (DT == 1) {
        x = pattern_value(w[0] & 0xffffu);
        w[0] = __builtin_amdgcn_alignbit(w[1], w[0], 16);
        w[1] = __builtin_amdgcn_alignbit(w[2], w[1], 16);
        w[2] = __builtin_amdgcn_alignbit(w[3], w[2], 16);
        w[3] >>= 16;
    } else {
        x = __uint_as_float(w[0]);
        w[0] = w[1];
        w[1] = w[2];
        w[2] = w[3];
    }
    return x;
}

// Weights under a cut law times a scale, computed from the logits.
template <int DT> struct DirectLaw {
    static constexpr int E = Elt<DT>::EPV;
    static constexpr bool AHEAD = true;
    RowCut r;
    double scale;
    __device__ __forceinline__ double one(float y, int id) const
    {
        return kept(order_key(y), id, r) && y != -INFINITY ? weight(y, r.max, r.c) * scale : 0.0;
    }
    __device__ __forceinline__ uint4 aux(int) const { return make_uint4(0, 0, 0, 0); }
    // float32: the weights of a group.  Its ids are all up to the last tie kept or all past it, so
    // one comparison tells, but for the group in which the kept ties end.
    __device__ __forceinline__ void four(int g, const uint4 &v, double (&w)[4]) const
    {
        const int id = g * 4;
        const float least = key_value(id <= r.tie ? r.cut : r.cut + 1);
        double a[4];
        unroll<0, 4>([&](auto k) SV_INLINE {
            const float x = __uint_as_float(vec_word(v, k));
            a[k] = ((double)(x >= least ? x : -INFINITY) - (double)r.max) * r.c;
        });
        if (__ballot(id <= r.tie && id + 3 > r.tie) != 0)
            unroll<0, 4>([&](auto k) SV_INLINE {
                if (!kept(order_key(__uint_as_float(vec_word(v, k))), id + k, r))
                    a[k] = -INFINITY;
            });
        exp2_neg4(a, w);
        unroll<0, 4>([&](auto k) SV_INLINE { w[k] *= scale; });
    }
    __device__ __forceinline__ double sum(int g, const uint4 &v, const uint4 &) const
    {
        double s = 0.0;
        if constexpr (DT == 0) {
            double x[4];
            four(g, v, x);
            unroll<0, 4>([&](auto k) SV_INLINE { s += x[k]; });
        } else {
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma nounroll
            for (int k = 0; k < E; ++k)
                s += one(next_logit<DT>(w), g * E + k);
        }
        return s;
    }
};

// The same from a table by bin, 0 for what the cut leaves out.
struct TableLaw {
    static constexpr bool AHEAD = true;
    RowCut r;
    double scale;
    const double *table;
    uint32_t cut_off;        // where some of the cut's ties are left out: its offset, if it has one
    bool low_counts;         // logits <= -2^8 may weigh something

    __device__ __forceinline__ TableLaw(const RowCut &c, int V, double sc, const double *tab)
        : r(uniform(c)), scale(uniform(sc)), table(tab), cut_off(~0u)
    {
        const uint32_t t = window_words(__float_as_uint(key_value(r.cut)) >> 16) & 0xffffu;
        if (r.tie < V && (t & 0x7000u) == 0)
            cut_off = offsets(t) & 0xffffu;
        low_counts = __builtin_amdgcn_readfirstlane(weight(-256.0f, r.max, r.c) >= 0x1p-80);
    }
    // How a unit's groups can be looked up: whole (no logit outside the window), with masked logits
    // left out, or id by id (rare values, low ones that count, and the group in which the kept ties
    // end).
    enum Way { WHOLE, MASKED, SINGLY };
    __device__ __forceinline__ Way by_table(int g, const uint4 &v, uint32_t (&t)[4]) const
    {
        uint32_t out = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            t[i] = window_words(vec_word(v, i));
            out |= t[i] & 0x70007000u;
        }
        if (__ballot(out != 0 || g == r.tie / 8) == 0)
            return WHOLE;
        uint32_t rare = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            rare |= rare_words(t[i], mask_words(vec_word(v, i)));
        return __ballot(rare != 0 || low_counts || g == r.tie / 8) == 0 ? MASKED : SINGLY;
    }
    // 8 * bin of both halves
    static __device__ __forceinline__ uint32_t offsets(uint32_t t)
    {
        const u16x2 three = {3, 3};
        return as_u32(as_u16x2(t) << three) | (t & 0x80008000u);
    }
    __device__ __forceinline__ double at(uint32_t off) const
    {
        return *reinterpret_cast<const double *>(reinterpret_cast<const char *>(table) + off);
    }
    // what a group past the last kept tie must not look up
    __device__ __forceinline__ uint32_t left_out(int g) const { return g > r.tie / 8 ? cut_off : ~0u; }
    __device__ __forceinline__ double at(uint32_t off, uint32_t without) const
    {
        const double x = at(off);
        return off == without ? 0.0 : x;
    }
    // the halves of window word t, 0 outside the window
    __device__ __forceinline__ double low_half(uint32_t t, uint32_t without) const
    {
        const double x = at(offsets(t) & 0xffffu, without);
        return (t & 0x7000u) == 0 ? x : 0.0;
    }
    __device__ __forceinline__ double high_half(uint32_t t, uint32_t without) const
    {
        const double x = at(offsets(t) >> 16, without);
        return (t & 0x70000000u) == 0 ? x : 0.0;
    }
    __device__ __forceinline__ double one(float y, int id) const
    {
        const uint32_t p = __float_as_uint(y) >> 16, t = window_words(p) & 0xffffu;
        if ((t & 0x7000u) == 0)
            return y == key_value(r.cut) && id > r.tie ? 0.0 : at(offsets(t) & 0xffffu);
        return kept(order_key(y), id, r) && y > (low_counts ? -INFINITY : -256.0f)
                   ? weight(y, r.max, r.c) * scale
                   : 0.0;
    }
    __device__ __forceinline__ uint4 aux(int) const { return make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ double sum(int g, const uint4 &v, const uint4 &) const
    {
        uint32_t t[4];
        double s = 0.0;
        const Way way = by_table(g, v, t);
        if (way == WHOLE) {
            if (cut_off == ~0u) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t b = offsets(t[i]);
                    s += at(b & 0xffffu);
                    s += at(b >> 16);
                }
            } else {
                const uint32_t no = left_out(g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t b = offsets(t[i]);
                    s += at(b & 0xffffu, no);
                    s += at(b >> 16, no);
                }
            }
        } else if (way == MASKED) {
            const uint32_t no = left_out(g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s += low_half(t[i], no);
                s += high_half(t[i], no);
            }
        } else {
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma nounroll
            for (int k = 0; k < 8; ++k)
                s += one(next_logit<1>(w), g * 8 + k);
        }
        return s;
    }
};

// max(0, p - q) of two laws' weights; the second operand of sum() is q's group.
template <int DT, typename P> struct ResidualLaw {
    static constexpr int E = Elt<DT>::EPV;
    static constexpr bool AHEAD = false;     // two rows: the registers hold one batch of each
    P p, q;
    Groups<DT> gq;
    bool both;                     // false: p alone
    __device__ __forceinline__ double one(float y, int id) const
    {
        const double x = p.one(y, id);
        return x > 0.0 && !both ? x : x > 0.0 ? fmax(x - q.one(Elt<DT>::one(gq.row, id), id), 0.0) : 0.0;
    }
    __device__ __forceinline__ uint4 aux(int g) const
    {
        return both ? gq.load(g) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ double sum(int g, const uint4 &pv, const uint4 &qv) const
    {
        double s = 0.0;
        if (!both)
            return p.sum(g, pv, qv);
        if constexpr (DT == 1) {
            uint32_t tp[4], tq[4];
            const auto a = p.by_table(g, pv, tp);
            const auto b = q.by_table(g, qv, tq);
            if (a == P::WHOLE && b == P::WHOLE) {
                const uint32_t np = p.left_out(g), nq = q.left_out(g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t op = P::offsets(tp[i]), oq = P::offsets(tq[i]);
                    s += fmax(p.at(op & 0xffffu, np) - q.at(oq & 0xffffu, nq), 0.0);
                    s += fmax(p.at(op >> 16, np) - q.at(oq >> 16, nq), 0.0);
                }
                return s;
            }
            if (a != P::SINGLY && b != P::SINGLY) {
                const uint32_t np = p.left_out(g), nq = q.left_out(g);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s += fmax(p.low_half(tp[i], np) - q.low_half(tq[i], nq), 0.0);
                    s += fmax(p.high_half(tp[i], np) - q.high_half(tq[i], nq), 0.0);
                }
                return s;
            }
        }
        uint32_t wp[4] = {pv.x, pv.y, pv.z, pv.w}, wq[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma nounroll
        for (int k = 0; k < E; ++k) {
            const float yp = next_logit<DT>(wp), yq = next_logit<DT>(wq);
            const double x = p.one(yp, g * E + k);
            if (x > 0.0)
                s += fmax(x - q.one(yq, g * E + k), 0.0);
        }
        return s;
    }
};

// table[bin] = w / z for the bins that r keeps, 0 for the others.
__device__ __forceinline__ void fill_table(const RowCut &r, double scale, double *table)
{
    const float low = key_value(r.cut);
    for (int b = threadIdx.x; b < HBINS; b += FWG) {
        const float x = pattern_value(bin_pattern(b));
        table[b] = x >= low && x <= r.max ? weight(x, r.max, r.c) * scale : 0.0;
    }
}

// One row: its cut by counting, then the draw.  256 rows of 128256 take 35 us without a cut, 27 with
// top-k or min-p, 47 with top-p and 43 with mixed parameters.  A workgroup's phases in us, the logits
// from the last-level cache: without a cut 7 to count, 7 for the cut (barriers and scans, one after
// the other), 13 for the sums, a second reading through the table (an 8-byte LDS lookup per logit,
// 12 clocks for a wave's, is what bounds it), 3 to find the id.  The slowest rows of the mixed batch
// are cut by top-p inside a run of equals and have no list: 6, 9, then 9 to find the last kept of
// the equals (a reading of its own), 13 and 3.  Rows cut by top-k or min-p list the groups that can
// matter while they count: 12, 5, up to 3, 2 and 2.  One row of 32000: 14 us, all of it latency.
__global__ __launch_bounds__(FWG, 4) void k_filter_sample_bf16(const char *logits, int V,
                                                               int64_t stride, FilterPtrs f,
                                                               const float *unif, int *tok,
                                                               float *prob)
{
    __shared__ __align__(16) uint32_t hist[HBINS];
    __shared__ __align__(16) double table[HBINS];
    __shared__ CutLds c;
    __shared__ DrawLds dl;
    __shared__ RedLds red;
    const int n = blockIdx.x;
    const char *row = logits + (size_t)n * stride * 2;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const Groups<1> gr(row, V);
    const Units<1> all{gr, nullptr, -1};
    uint4 nx[BATCH];
    load_batch(all, 0, nx);
    const Params q = load_params(f, n, V);
    Floor fl(q, V, FWAVES);
    clear_hist<FWG>(hist);
    if (fl.active())                       // what is not counted is looked up all the same
        for (int b = threadIdx.x; b < HBINS / 2; b += FWG)
            reinterpret_cast<double2 *>(table)[b] = make_double2(0.0, 0.0);
    cut_lds_clear(c);
    __syncthreads();
    int listed = 0;
    uint32_t low = NO_LOW;
    const int units = all.count(), trips = fl.active() ? gr.per_wave : units;
#pragma nounroll
    for (int i0 = 0; i0 < trips; i0 += BATCH) {
        uint4 v[BATCH];
        unroll<0, BATCH>([&](auto j) SV_INLINE { v[j] = nx[j]; });
        if (i0 + BATCH < trips)
            load_batch(all, i0 + BATCH, nx);
        if (fl.active()) {
            unroll<0, BATCH>([&](auto j) SV_INLINE { fl.see(v[j]); });
            fl.exchange<FWAVES>(c, i0 / BATCH);
        }
        if (fl.below == 0) {
            listed = LIST + 1;
            unroll<0, BATCH>([&](auto j) SV_INLINE {
                if (i0 + j < units)
                    count_vec(v[j], hist, c, low);
            });
        } else {
            unroll<0, BATCH>([&](auto j) SV_INLINE {
                const bool m = i0 + j < units && fl.matters(v[j]);
                list_groups(dl.list[wv], listed, m, (i0 + j) * 64 + lane);
                if (m)
                    count_vec(v[j], hist, c, low);
            });
        }
    }
    note_low(low, c);
    if (fl.active() && fl.bad())
        atomicOr(&c.bad, 1u);
    cut_from_counts<FWG>(hist, c, q, V, !fl.active(), table);
    RowCut r = c.cut;
    int id = -1;
    const double u = (double)unif[n];
    if (r.state == CUT_EXACT) {
        r = cut_by_bisection<1>(row, V, q, red);
        if (r.state == CUT_READY)
            id = draw_row(all, MayKeep<1>(r), u, dl, DirectLaw<1>{r, 1.0});
    } else if (r.state != CUT_NONE) {
        const Units<1> few{gr, dl.list[wv], listed <= LIST ? __builtin_amdgcn_readfirstlane(listed) : -1};
        if (r.state == CUT_TIES)
            find_ties(few, few, 1, r, r, dl);
        id = draw_row(few, MayKeep<1>(r), u, dl, TableLaw(r, V, 1.0, table));
    }
    if (threadIdx.x == 0) {
        tok[n] = id;
        if (prob)
            prob[n] = id < 0 ? NAN : (float)(weight(Elt<1>::one(row, id), r.max, r.c) / r.z);
    }
}

// ------------------------------------------------------------------ float32: the cut by counting
//
// The upper halves of float32 logits are counted in the bins of the bfloat16 path (truncated, which
// keeps the order), with three more for what lies above, around zero and below.  The counts name
// the bin of a cut; the few logits of that bin, or of it and all above, are then gathered and put
// in order exactly.  For top-p the bins' weights are needed too: one more pass adds them up in
// LDS, as integers so that their order does not matter, in units of 2^-47 (for vocabularies past
// 2^15 coarser, 2^-41 at 2^20) of the weight at the bin's upper edge.  Half a unit is lost per logit
// at most, so V halves of a unit of a row's sum at worst: 2^-33 up to 2^15 ids, 2^-28 at 2^17.  The
// errors of a row's logits have no sign in common, which leaves about one unit.  A bin of more than
// GATHER logits is counted once more by its next 13 bits.  A row in which even that leaves more,
// GATHER equal logits at its cut, goes to cut_by_bisection.

constexpr int BIN_HIGH = HBINS, BIN_ZERO = HBINS + 1, BIN_LOW = HBINS + 2, FBINS = HBINS + 3;
constexpr int GATHER = 1024;
// Where top-k keeps little, all of it is put in order at once instead of its last bin alone: that
// spares the sum over the row that gives Z, and with top-p the weights' pass, but an order of n
// costs n comparisons of each.  The cuts of 576 rows of 32000 in us, at once and by the bin: k = 20
// 46.7 and 47.8, 50 49.9 and 48.9, 250 63 and 51; with top-p k = 50 50 and 74, 400 77 and 85, 800
// 118 and 101.
constexpr int AT_ONCE = 32, AT_ONCE_P = 512;

struct FloatLds {
    __align__(16) uint32_t hist[FBINS + 1];
    unsigned long long weight[FBINS];
    unsigned long long list[GATHER], order[GATHER];   // order key, then ~id
    double dwave[FWAVES];
    double prefix;                 // what find_bin found
    int bin, place;
    uint32_t n;
};

// Which logits a bin holds: from low() to high().
__device__ __forceinline__ float bin_low(int bin)
{
    if (bin >= HBINS)
        return bin == BIN_HIGH ? 256.0f : bin == BIN_ZERO ? -__uint_as_float((HLO << 16) - 1) : -FLT_MAX;
    const uint32_t p = bin_pattern(bin);
    return __uint_as_float(p << 16 | (bin >= HMAG ? 0xffffu : 0u));
}
__device__ __forceinline__ float bin_high(int bin)
{
    if (bin >= HBINS)
        return bin == BIN_HIGH ? FLT_MAX : bin == BIN_ZERO ? __uint_as_float((HLO << 16) - 1) : -256.0f;
    const uint32_t p = bin_pattern(bin);
    return __uint_as_float(p << 16 | (bin >= HMAG ? 0u : 0xffffu));
}

// The bin of a finite logit.
__device__ __forceinline__ int float_bin(uint32_t bits)
{
    const uint32_t t = ((bits >> 16) - HLO) & 0xffffu;
    if ((t & 0x7000u) == 0)
        return (int)((t >> 15) * HMAG + (t & 0xfffu));
    return (bits & 0x7fffffffu) < HLO << 16 ? BIN_ZERO : bits >> 31 ? BIN_LOW : BIN_HIGH;
}

// Upper halves of four float32 words, two to a word.
__device__ __forceinline__ uint2 upper_halves(const uint4 &v)
{
    return make_uint2(__builtin_amdgcn_perm(v.y, v.x, 0x07060302u),
                      __builtin_amdgcn_perm(v.w, v.z, 0x07060302u));
}

// Masked logits are left out, the finite ones counted in `low` by each lane.
__device__ __forceinline__ bool outside(const uint2 &h)
{
    return ((window_words(h.x) | window_words(h.y)) & 0x70007000u) != 0;
}

__device__ __forceinline__ void count_inside(const uint2 &h, uint32_t *hist)
{
    const uint32_t a = bin_offsets(window_words(h.x)), b = bin_offsets(window_words(h.y));
    bump(hist, a & 0xffffu);
    bump(hist, a >> 16);
    bump(hist, b & 0xffffu);
    bump(hist, b >> 16);
}

__device__ __forceinline__ void count_any(const uint4 &v, const uint2 &h, FloatLds &f, CutLds &c,
                                          uint32_t &low)
{
    const uint32_t t0 = window_words(h.x), t1 = window_words(h.y);
    const uint32_t a = bin_offsets(t0), b = bin_offsets(t1);
    if ((t0 & 0x7000u) == 0)
        bump(f.hist, a & 0xffffu);
    if ((t0 & 0x70000000u) == 0)
        bump(f.hist, a >> 16);
    if ((t1 & 0x7000u) == 0)
        bump(f.hist, b & 0xffffu);
    if ((t1 & 0x70000000u) == 0)
        bump(f.hist, b >> 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    unroll<0, 4>([&](auto k) SV_INLINE { low += w[k] - (MASK_TOP << 16) < MASK_INF << 16; });
    if (__ballot((rare_words(t0, mask_words(h.x)) | rare_words(t1, mask_words(h.y))) != 0) != 0) {
        uint32_t w0 = v.x, w1 = v.y, w2 = v.z, w3 = v.w;
#pragma nounroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = w0 >> 16;
            if (rare_words(window_words(u), mask_words(u)) & 0xffffu) {
                if ((w0 & 0x7f800000u) != 0x7f800000u)
                    atomicAdd(&f.hist[float_bin(w0)], 1u);
                else
                    atomicOr(&c.bad, 1u);
            }
            w0 = w1;
            w1 = w2;
            w2 = w3;
        }
    }
}

// The workgroup's inclusive scan in thread order; *total is the sum.
__device__ __forceinline__ double block_scan(double v, double *lds, double *total)
{
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    v = wave_incl_scan(v);
    __syncthreads();
    if (lane == 63)
        lds[wv] = v;
    __syncthreads();
    const double w = lane < FWAVES ? lds[lane] : 0.0, wi = wave_incl_scan(w);
    *total = lane_value(wi, 63);
    return lane_value(wave_excl_from_incl(wi), __builtin_amdgcn_readfirstlane(wv)) + v;
}

// The last bin, in order, that holds something and before which (counting `base` before all) lies
// less than goal; f.bin and f.prefix.  val(bin) is what a bin holds, goal_of(total) the goal.
// Returns the total.  A thread takes eight bins; those outside the window join the threads that
// they stand next to.  SUB: the bins are parts of one, by magnitude; `down`: the largest first.
template <bool SUB, typename W, typename G>
__device__ __forceinline__ double find_bin(FloatLds &f, double base, bool down, W val, G goal_of)
{
    const int t = threadIdx.x;
    constexpr int PER = HBINS / FWG;
    auto bin_of = [&](int i) SV_INLINE {       // i = 0: before the eight, 9: after them
        const int o = t * PER + i - 1;
        if (i == 0)
            return SUB ? -1 : t == 0 ? BIN_HIGH : t == FWG / 2 ? BIN_ZERO : -1;
        if (i == PER + 1)
            return !SUB && t == FWG - 1 ? BIN_LOW : -1;
        if (SUB)
            return down ? HBINS - 1 - o : o;
        return o < HMAG ? HMAG - 1 - o : o;
    };
    double v[PER + 2], sum = 0.0, total;
    if (t == 0)
        f.place = -1;
    unroll<0, PER + 2>([&](auto i) SV_INLINE {
        const int b = bin_of(i);
        v[i] = b >= 0 ? val(b) : 0.0;
        sum += v[i];
    });
    const double inc = block_scan(sum, f.dwave, &total), goal = goal_of(total);
    double run = __shfl_up(inc, 1);            // what stands before the thread
    if ((t & 63) == 0) {
        run = 0.0;
        for (int i = 0; i < t >> 6; ++i)
            run += f.dwave[i];
    }
    run += base;
    if (sum > 0.0 && run < goal)
        atomicMax(&f.place, t);
    __syncthreads();
    if (f.place == t)
        unroll<0, PER + 2>([&](auto i) SV_INLINE {
            if (v[i] > 0.0 && run < goal) {
                f.bin = bin_of(i);
                f.prefix = run;
            }
            run += v[i];
        });
    __syncthreads();
    return total;
}

// Runs f(four logits' bits, the first's id) over the wave's units, -inf where there are none; all
// lanes together.
template <typename F> __device__ __forceinline__ void each_vec(const Units<0> &un, F f)
{
    const int units = un.count();
#pragma nounroll
    for (int i0 = 0; i0 < units; i0 += BATCH) {
        uint4 v[BATCH];
        load_batch(un, i0, v);
#pragma nounroll
        for (int j = 0; j < BATCH && i0 + j < units; ++j) {
            uint4 x = choose(v, j);
            if (!un.holds(i0 + j))
                x = make_uint4(un.gr.EMPTY, un.gr.EMPTY, un.gr.EMPTY, un.gr.EMPTY);
            f(x, un.group(i0 + j) * 4);
        }
    }
}

// Runs f(bits, id) over the logits from lo to hi that r keeps.
template <typename F>
__device__ __forceinline__ void each_between(const Units<0> &un, float lo, float hi, const RowCut &r, F f)
{
    each_vec(un, [&](const uint4 &v, int id) SV_INLINE {
        auto in = [&](uint32_t w) SV_INLINE { return __uint_as_float(w) >= lo && __uint_as_float(w) <= hi; };
        if (__ballot(in(v.x) || in(v.y) || in(v.z) || in(v.w)) == 0)
            return;
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma nounroll
        for (int k = 0; k < 4; ++k) {
            if (in(w[0]) && kept(order_key(__uint_as_float(w[0])), id + k, r))
                f(w[0], id + k);
            w[0] = w[1];
            w[1] = w[2];
            w[2] = w[3];
        }
    });
}

// The logits from lo to hi that r keeps, gathered and put in order: f.order[0 .. f.n).  False if
// there are too many.
__device__ __forceinline__ bool gather(const Units<0> &un, float lo, float hi, const RowCut &r, FloatLds &f)
{
    if (threadIdx.x == 0)
        f.n = 0;
    __syncthreads();
    each_between(un, lo, hi, r, [&](uint32_t bits, int id) SV_INLINE {
        const uint32_t at = atomicAdd(&f.n, 1u);
        if (at < GATHER)
            f.list[at] = (unsigned long long)order_key(__uint_as_float(bits)) << 32 | (uint32_t)~id;
    });
    __syncthreads();
    const int n = (int)f.n;
    if (n > GATHER)
        return false;
    if ((int)threadIdx.x < n) {
        const unsigned long long me = f.list[threadIdx.x];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j)
            rank += f.list[j] > me;
        f.order[rank] = me;
    }
    __syncthreads();
    return true;
}

// What the logits from lo to hi, a bin's, that r keeps hold by their next 13 bits: of(x) each, in
// f.weight.
template <typename O>
__device__ __forceinline__ void count_parts(const Units<0> &un, float lo, float hi, const RowCut &r,
                                            FloatLds &f, O of)
{
    for (int i = threadIdx.x; i < HBINS; i += FWG)
        f.weight[i] = 0;
    __syncthreads();
    each_between(un, lo, hi, r, [&](uint32_t bits, int) SV_INLINE {
        atomicAdd(&f.weight[(bits & 0xffffu) >> 3], of(__uint_as_float(bits)));
    });
    __syncthreads();
}

__device__ __forceinline__ void part_range(int bin, int part, float &lo, float &hi)
{
    const uint32_t p = bin_pattern(bin) << 16 | (uint32_t)part << 3;
    lo = __uint_as_float(bin >= HMAG ? p | 7u : p);
    hi = __uint_as_float(bin >= HMAG ? p : p | 7u);
}

// How many of the ordered logits, of which there is one at least, stay: those before which less than
// goal lies (counting `base` before all of them), of weight at least m and among the first k; with
// p < 1 the goal is p times the sum over the first k.  Sets r's cut to the last, and its z.
__device__ __forceinline__ void cut_in_order(RowCut &r, double base, int k, double p, double goal,
                                             double m, FloatLds &f)
{
    const int t = threadIdx.x, n = min((int)f.n, k);
    const double w = t < n ? weight(key_value((uint32_t)(f.order[t] >> 32)), r.max, r.c) : 0.0;
    double total;
    const double inc = block_scan(w, f.dwave, &total);
    if (p < 1.0)
        goal = p * total;
    // the exclusive prefix as the sum of what stands before, not the difference with w
    const double left = __shfl_up(inc, 1);
    double before = left;
    if ((t & 63) == 0) {
        before = 0.0;
        for (int i = 0; i < t >> 6; ++i)
            before += f.dwave[i];
    }
    before += base;
    // the first stays whatever the rounding: it is the row's largest, or m is 0
    const bool keep = t < n && (t == 0 || (before < goal && w >= m));
    const int stay = __syncthreads_count(keep);
    if (t == stay - 1) {
        f.place = (int)~(uint32_t)f.order[t];
        f.dwave[0] = base + inc;
    }
    __syncthreads();
    r.cut = (uint32_t)(f.order[stay - 1] >> 32);
    r.tie = f.place;
    r.z = f.dwave[0];
    r.kept = stay;
    __syncthreads();
}

// The lowest key of weight at least m, 64 at a time.
__device__ __forceinline__ uint32_t key_of_weight(float M, double c, double m)
{
    uint32_t lo = KEY_NEG_INF, hi = order_key(M);     // weight(hi) >= m
#pragma nounroll
    while (lo < hi) {
        const uint32_t step = (hi - lo) / 64 + 1, lane = threadIdx.x & 63;
        const uint32_t key = hi - lo < lane * step ? hi : lo + lane * step;
        const unsigned long long ok = __ballot(weight(key_value(key), M, c) >= m);
        const int l = ok ? __ffsll(ok) - 1 : 64;       // the first of the probes that passes
        const uint32_t up = l == 64 || hi - lo < (uint32_t)l * step ? hi : lo + (uint32_t)l * step;
        lo = l == 0 ? lo : min(lo + (uint32_t)(l - 1) * step + 1, up);
        hi = up;
        if (l == 0)
            break;
    }
    return hi;
}

// A float32 row's cut.  few receives the units that hold what matters.  z is left at 0 where only
// a sum over the kept ids would give it.
__device__ __forceinline__ RowCut cut_floats(const Units<0> &all, Units<0> &few, const Params &q, FloatLds &f,
                                             CutLds &c, DrawLds &dl, RedLds &red)
{
    const int t = threadIdx.x, lane = t & 63, wv = t >> 6, V = all.gr.V, units = all.count();
    for (int i = t; i < FBINS; i += FWG)
        f.hist[i] = 0;
    cut_lds_clear(c);
    __syncthreads();
    Floor fl(q, V, FWAVES);
    float mx = -INFINITY;
    uint32_t most = 0;             // as unsigned bits: a NaN of negative sign is above -inf
    uint32_t low = 0;              // finite logits <= -2^8
    int listed = 0;
    const int trips = fl.active() ? all.gr.per_wave : units;
#pragma nounroll
    for (int i0 = 0; i0 < trips; i0 += BATCH) {
        uint4 v[BATCH];
        uint2 h[BATCH];
        load_batch(all, i0, v);
        unroll<0, BATCH>([&](auto j) SV_INLINE {
            h[j] = upper_halves(v[j]);
            mx = fmaxf(fmaxf(mx, fmaxf(__uint_as_float(v[j].x), __uint_as_float(v[j].y))),
                       fmaxf(__uint_as_float(v[j].z), __uint_as_float(v[j].w)));
            most = max(max(most, max(v[j].x, v[j].y)), max(v[j].z, v[j].w));
        });
        if (fl.active()) {
            unroll<0, BATCH / 2>([&](auto j) SV_INLINE {
                fl.see(make_uint4(h[2 * j].x, h[2 * j].y, h[2 * j + 1].x, h[2 * j + 1].y));
            });
            fl.exchange<FWAVES>(c, i0 / BATCH);
        }
        uint32_t wait = 0;
        auto matters = [&](const uint2 &x) SV_INLINE {
            return max_i16(max_i16(x.x, x.y), fl.below) != fl.below;
        };
        if (fl.below == 0) {
            listed = LIST + 1;
            unroll<0, BATCH>([&](auto j) SV_INLINE {
                if (i0 + j < units) {
                    if (__ballot(outside(h[j])) == 0)
                        count_inside(h[j], f.hist);
                    else
                        wait |= 1u << j;
                }
            });
        } else {
            unroll<0, BATCH>([&](auto j) SV_INLINE {
                const bool m = i0 + j < units && matters(h[j]);
                list_groups(dl.list[wv], listed, m, (i0 + j) * 64 + lane);
                if (__ballot(m && outside(h[j])) != 0)
                    wait |= 1u << j;
                else if (m)
                    count_inside(h[j], f.hist);
            });
        }
#pragma nounroll
        for (wait = __builtin_amdgcn_readfirstlane(wait); wait; wait &= wait - 1) {
            const uint4 x = choose(v, __builtin_ctz(wait));
            const uint2 y = upper_halves(x);
            if (fl.below == 0 || matters(y))
                count_any(x, y, f, c, low);
        }
    }
    if (most > 0xff800000u)
        atomicOr(&c.bad, 1u);
    if (__ballot(low != 0) != 0) {
        low = wave_scan_u32(low);
        if (lane == 63)
            atomicAdd(&f.hist[BIN_LOW], low);
    }
    few.n = listed <= LIST ? __builtin_amdgcn_readfirstlane(listed) : -1;
    few.list = dl.list[wv];
    RowCut r;
    r.max = key_value(block_max(order_key(mx), red.u));       // and the counts are complete
    r.c = q.c;
    r.cut = KEY_NEG_INF;
    r.tie = V;
    r.z = 0.0;
    r.kept = V;
    r.state = q.ok && !c.bad && r.max != -INFINITY ? CUT_READY : CUT_NONE;
    if (r.state == CUT_NONE)
        return r;
    if (q.k < V) {
        // what min-p's floor passed over was not counted: then fewer than k may be left
        double total = 0.0;
        find_bin<false>(f, 0.0, false, [&](int b) SV_INLINE { return (double)f.hist[b]; },
                        [&](double n) SV_INLINE {
                            total = n;
                            return fmin((double)q.k, n);
                        });
        if (fl.active() || (double)q.k < total) {
            const int k = (int)fmin((double)q.k, total);
            const int bin = f.bin;
            uint32_t before = (uint32_t)f.prefix;
            float lo = bin_low(bin), hi = bin_high(bin);
            // What min-p's floor passed over is not in the counts but may be met again below, where
            // a wave has no list.  All of it lies below this bound, and nothing there is kept.
            const float least = fl.by_m ? r.max + fl.drop : -INFINITY;
            const bool some = hi >= least;
            if (some && before + f.hist[bin] <= (q.p < 1.0 ? AT_ONCE_P : AT_ONCE)) {
                // all that top-k can keep is in hand: the three cuts at once
                if (gather(few, fmaxf(lo, least), FLT_MAX, r, f))
                    cut_in_order(r, 0.0, q.k, q.p, INFINITY, q.m, f);
                else
                    r.state = CUT_EXACT;
                return r;
            }
            if (some && f.hist[bin] > GATHER && bin < HBINS) {
                const double was = f.prefix;
                count_parts(few, fmaxf(lo, least), hi, r, f, [&](float) SV_INLINE { return 1ull; });
                find_bin<true>(f, was, bin < HMAG, [&](int b) SV_INLINE { return (double)f.weight[b]; },
                               [&](double) SV_INLINE { return (double)k; });
                before = (uint32_t)f.prefix;
                part_range(bin, f.bin, lo, hi);
            }
            if (some && !gather(few, fmaxf(lo, least), hi, r, f)) {
                r.state = CUT_EXACT;
                return r;
            }
            // where the k-th lies below the bound, min-p alone cuts the row
            if (some && k - (int)before <= (int)f.n) {
                const unsigned long long last = f.order[k - before - 1];
                r.cut = (uint32_t)(last >> 32);
                r.tie = (int)~(uint32_t)last;
            }
            r.kept = k;            // at most: what a draw decides by
            __syncthreads();
        }
    }
    if (q.p < 1.0) {
        const double unit = ldexp(1.0, min(47, 62 - (32 - __clz(V))));
        const bool cut = r.cut != KEY_NEG_INF;     // then the counts are those of the kept, once more
        for (int i = t; i < FBINS; i += FWG) {
            f.weight[i] = 0;
            if (cut)
                f.hist[i] = 0;
        }
        __syncthreads();
        // no edge lies above the maximum, so that its own weight is 1
        auto edge = [&](int b) SV_INLINE { return fminf(bin_high(b), r.max); };
        // a weight, w * unit to the nearest integer, in the low bits of the sum with 2^52
        auto to_units = [&](double w) SV_INLINE {
            return (unsigned long long)__double_as_longlong(fma(w, unit, 0x1p52)) & 0xfffffffffffffull;
        };
        const float small = (float)(-0.249 / r.c);      // in logits, what exp2_small takes
        auto units_of = [&](float x, float top) SV_INLINE { return to_units(weight(x, top, r.c)); };
        // the sums in units to weights in place, each where its bin's neighbours are other threads'
        auto weigh = [&](int bins, auto top) SV_INLINE {
#pragma nounroll
            for (int b = t; b < bins; b += FWG) {
                const unsigned long long n = f.weight[b];
                if (n)
                    f.weight[b] = (unsigned long long)__double_as_longlong(
                        (double)n * (1.0 / unit) * weight(top(b), r.max, r.c));
            }
            __syncthreads();
        };
        auto weight_of = [&](int b) SV_INLINE { return __longlong_as_double((long long)f.weight[b]); };
        // masked logits are passed over where even V of -2^8 would not be noticed
        const bool low_counts = weight(edge(BIN_LOW), r.max, r.c) >= 0x1p-80;
        each_vec(few, [&](const uint4 &v, int id) SV_INLINE {
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
            const uint2 h = upper_halves(v);
            const uint32_t t0 = window_words(h.x), t1 = window_words(h.y);
            const uint32_t other = low_counts ? (t0 | t1) & 0x70007000u
                                              : rare_words(t0, mask_words(h.x)) | rare_words(t1, mask_words(h.y));
            if (__ballot(other != 0) == 0) {
                // all in the window, or masked, whose weights come to nothing of use.  An edge is
                // the logit's own upper half, and their difference is exact, since they share an
                // exponent.
                const bool whole = __ballot(((t0 | t1) & 0x70007000u) != 0) == 0;
                const uint32_t out[4] = {t0 & 0x7000u, t0 & 0x70000000u, t1 & 0x7000u, t1 & 0x70000000u};
                float d[4];
                double a[4], p[4];
                unroll<0, 4>([&](auto k) SV_INLINE {
                    const uint32_t e = (w[k] & 0xffff0000u) | (~(uint32_t)((int32_t)w[k] >> 31) & 0xffffu);
                    d[k] = __uint_as_float(w[k]) - fminf(__uint_as_float(e), r.max);
                    a[k] = (double)d[k] * r.c;
                });
                if (__ballot(fminf(fminf(d[0], d[1]), fminf(d[2], d[3])) < small) == 0)
                    unroll<0, 4>([&](auto k) SV_INLINE { p[k] = exp2_small(a[k]); });
                else
                    exp2_neg4(a, p);
                const uint32_t b0 = bin_offsets(t0), b1 = bin_offsets(t1);
                const uint32_t at[4] = {b0 & 0xffffu, b0 >> 16, b1 & 0xffffu, b1 >> 16};
                unroll<0, 4>([&](auto k) SV_INLINE {
                    if (!whole && out[k] != 0)
                        return;
                    if (cut && !kept(order_key(__uint_as_float(w[k])), id + k, r))
                        return;
                    atomicAdd(&f.weight[at[k] / 4], to_units(p[k]));
                    if (cut)
                        atomicAdd(&f.hist[at[k] / 4], 1u);
                });
            } else {
#pragma nounroll
                for (int k = 0; k < 4; ++k) {
                    const float x = __uint_as_float(w[0]);
                    if (x > (low_counts ? -INFINITY : -256.0f) && kept(order_key(x), id + k, r)) {
                        const int b = float_bin(w[0]);
                        atomicAdd(&f.weight[b], units_of(x, edge(b)));
                        if (cut)
                            atomicAdd(&f.hist[b], 1u);
                    }
                    w[0] = w[1];
                    w[1] = w[2];
                    w[2] = w[3];
                }
            }
        });
        __syncthreads();
        weigh(FBINS, edge);
        double goal = 0.0;
        find_bin<false>(
            f, 0.0, false, weight_of,
            [&](double z) SV_INLINE {
                goal = q.p * z;
                return fmax(goal, 0x1p-1074);  // the first bin at least
            });
        const int bin = f.bin;
        const float top = edge(bin);
        double base = f.prefix;
        float lo = bin_low(bin), hi = bin_high(bin);
        if (bin < HBINS && f.hist[bin] > GATHER) {
            __syncthreads();
            count_parts(few, lo, hi, r, f, [&](float x) SV_INLINE { return units_of(x, top); });
            weigh(HBINS, [&](int) SV_INLINE { return top; });
            find_bin<true>(f, base, bin < HMAG, weight_of,
                           [&](double) SV_INLINE { return fmax(goal, 0x1p-1074); });
            base = f.prefix;
            part_range(bin, f.bin, lo, hi);
        }
        if (!gather(few, lo, hi, r, f)) {
            r.state = CUT_EXACT;
            return r;
        }
        const int kept_at_most = r.kept;
        cut_in_order(r, base, GATHER, 1.0, goal, 0.0, f);
        r.kept = kept_at_most;
    }
    if (q.m > 0.0 && weight(key_value(r.cut), r.max, r.c) < q.m) {
        r.cut = key_of_weight(r.max, r.c, q.m);
        r.tie = V;
        r.z = 0.0;
    }
    return r;
}

// The kept weight of a whole row, the same bits in every thread.
template <int DT, typename W>
__device__ __forceinline__ double row_total(const Units<DT> &un, const MayKeep<DT> &may, const W &law,
                                            RedLds &red)
{
    const int units = un.count();
    double s = 0.0;
#pragma nounroll
    for (int i0 = 0; i0 < units; i0 += BATCH) {
        uint4 v[BATCH], x[BATCH];
        load_batch(un, i0, v);
        const uint32_t mask = look(un, i0, v, x, may, law);
        unroll<0, BATCH>([&](auto j) SV_INLINE {
            if (mask >> j & 1) {
                const double w = law.sum(un.group(i0 + j), v[j], x[j]);
                s += un.holds(i0 + j) ? w : 0.0;
            }
        });
    }
    return block_sum(s, red.d);
}

// One row.  64 rows of 32000 with top-p alone, which skips nothing, take 48 us, the time of the
// slowest.  Its workgroup's phases in us: counting 3, the maximum 2, the weights' pass 13 (fp64
// issue), the goal's bin 4, gathering and ordering its logits 9 (half of that in a median row), the
// cut 2, the draw's sums 9 and its search 3.  With top-k 21 us.
__global__ __launch_bounds__(FWG, 4) void k_filter_sample_f32(const char *logits, int V,
                                                              int64_t stride, FilterPtrs f,
                                                              const float *unif, int *tok,
                                                              float *prob)
{
    __shared__ FloatLds fl;
    __shared__ CutLds c;
    __shared__ DrawLds dl;
    __shared__ RedLds red;
    const int n = blockIdx.x;
    const char *row = logits + (size_t)n * stride * 4;
    const Groups<0> gr(row, V);
    const Units<0> all{gr, nullptr, -1};
    Units<0> few = all;
    const Params q = load_params(f, n, V);
    RowCut r = cut_floats(all, few, q, fl, c, dl, red);
    if (r.state == CUT_EXACT) {
        r = cut_by_bisection<0>(row, V, q, red);
        few.n = -1;
    }
    int id = -1;
    if (r.state == CUT_READY)
        id = draw_row(few, MayKeep<0>(r), (double)unif[n], dl, DirectLaw<0>{uniform(r), 1.0});
    if (threadIdx.x == 0) {
        tok[n] = id;
        if (prob) {
            const double z = r.z > 0.0 ? r.z : dl.total;
            prob[n] = id < 0 ? NAN : (float)(weight(Elt<0>::one(row, id), r.max, r.c) / z);
        }
    }
}

// The RowCut of every target and draft row of a float32 verify: the B (K+1) target rows, then the
// B K draft rows.  The counts, weights and lists take 131 KB of LDS, so a compute unit holds one
// workgroup and a row's phases wait for each other: 704 rows of 32000 with top-k take 48 us, three
// rounds of 16, where the bytes need 13.
__global__ __launch_bounds__(FWG, 4) void k_filter_rows_f32(const char *tgt, const char *drf, int B,
                                                            int K, int V, FilterPtrs ft,
                                                            FilterPtrs fd, RowCut *cuts)
{
    __shared__ FloatLds fl;
    __shared__ CutLds c;
    __shared__ DrawLds dl;
    __shared__ RedLds red;
    const int n = blockIdx.x, nt = B * (K + 1);
    const bool is_t = n < nt;
    const char *row = is_t ? tgt + (size_t)n * V * 4 : drf + (size_t)(n - nt) * V * 4;
    const Params q = is_t ? load_params(ft, n / (K + 1), V) : load_params(fd, (n - nt) / K, V);
    const Groups<0> gr(row, V);
    const Units<0> all{gr, nullptr, -1};
    Units<0> few = all;
    RowCut r = cut_floats(all, few, q, fl, c, dl, red);
    if (r.state == CUT_EXACT)
        r = cut_by_bisection<0>(row, V, q, red);
    else if (r.state == CUT_READY && r.z == 0.0)
        r.z = row_total(few, MayKeep<0>(r), DirectLaw<0>{uniform(r), 1.0}, red);
    if (threadIdx.x == 0)
        cuts[n] = r;
}

constexpr int MAX_POS = 63;
// A target row that keeps no more ids than this is drawn from by lists of its groups: 11/16 of the
// places that the waves' lists have, so that ids spread evenly do not overflow one.  256 sequences
// of 128256 in bfloat16, with lists and without: k = 50 42 and 50 us, 1000 47 and 64, 3000 58 and
// 63; 4000, where lists overflow, 79 and 66.  64 of 32000 in float32: k = 50 15 and 19, 3000 27 and
// 42.
constexpr uint32_t SPARSE = 2816;

struct VerifyLds {
    RowCut cut[2 * MAX_POS + 1];          // target rows 0..K, then draft rows 0..K-1
    double P[MAX_POS + 1], Q[MAX_POS + 1];
    unsigned long long look_p, look_q;    // positions whose draft id equals a partly kept cut
    int L;
};

// Accept tests, first rejection and the replacement or bonus draw of one sequence.  256 sequences of
// 128256 in bfloat16 take 60 us with mixed parameters, since a chip has as many workgroups in flight
// as sequences and a batch waits for its slowest.  Phases in us of such a one, whose p keeps much and
// whose cuts fall inside runs of equals: 4 for the tests (a draft id equal to a partly kept cut adds a
// reading of its row), 2 for the tables, 19 to find the last kept equals of both rows, 27 for the
// sums of p - q (two lookups per id, as in the sampler), 6 to find the id.  The median sequence, whose
// p keeps few: 4, 2, 11 to list p's groups, 4 and 3.
template <int DT>
__global__ __launch_bounds__(FWG, 4) void k_filter_verify(const char *tgt, const char *drf, int B,
                                                          int K, int V, FilterPtrs ft, FilterPtrs fd,
                                                          const int *tokens, const float *unif,
                                                          const RowCut *cuts, int *acc, int *out,
                                                          float *probs)
{
    __shared__ __align__(16) double tables[2][DT == 1 ? HBINS : 1];
    __shared__ VerifyLds s;
    __shared__ DrawLds dl;
    __shared__ RedLds red;
    const int b = blockIdx.x, t = threadIdx.x;
    const size_t rb = (size_t)V * Elt<DT>::BYTES;
    const char *trow = tgt + (size_t)b * (K + 1) * rb, *drow = drf + (size_t)b * K * rb;
    auto row_of = [&](int i) { return i <= K ? trow + i * rb : drow + (i - K - 1) * rb; };
    if (t < 2 * K + 1)
        s.cut[t] = t <= K ? cuts[(size_t)b * (K + 1) + t]
                          : cuts[(size_t)B * (K + 1) + (size_t)b * K + (t - K - 1)];
    __syncthreads();
    for (int i = 0; i < 2 * K + 1; ++i)
        if (s.cut[i].state == CUT_EXACT) {
            const RowCut r = cut_by_bisection<DT>(row_of(i), V, load_params(i <= K ? ft : fd, b, V), red);
            __syncthreads();
            if (t == 0)
                s.cut[i] = r;
            __syncthreads();
        }
    // lane j: position j.  A draft id equal to a cut that keeps some of its ties counts as kept
    // until its rank among them is known.
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
        const unsigned long long lp = __ballot(lookp), lq = __ballot(lookq);
        if (t == 0) {
            s.L = good ? 0 : -1;
            s.look_p = good ? lp : 0;
            s.look_q = good ? lq : 0;
        }
    }
    __syncthreads();
    for (int side = 0; side < 2; ++side)
        for (unsigned long long m = side ? s.look_q : s.look_p; m; m &= m - 1) {
            const int j = __ffsll(m) - 1, i = side ? K + 1 + j : j;
            const int n = equals_below(Groups<DT>(row_of(i), V), tokens[(size_t)b * K + j],
                                       key_value(s.cut[i].cut), red);
            if (t == 0 && n >= s.cut[i].tie)
                (side ? s.Q : s.P)[j] = 0.0;
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
        // p's row, and q's where there is one
        const Groups<DT> gp(row_of(L), V), gq(row_of(L < K ? K + 1 + L : L), V);
        const Units<DT> uq{gq, nullptr, -1};
        Units<DT> up{gp, nullptr, -1};
        RowCut rp = s.cut[L], rq = s.cut[L < K ? K + 1 + L : L];
        if constexpr (DT == 1)
#pragma nounroll
            for (int side = 0; side < (L < K ? 2 : 1); ++side)
                fill_table(side ? rq : rp, 1.0 / (side ? rq : rp).z, tables[side]);
        // Where p keeps few ids, one pass over p lists their groups and the rest looks at those
        // alone.  q's last kept tie matters only if one of them has q's cut value.
        const bool sparse = rp.kept <= SPARSE;
        int need = (rp.state == CUT_TIES ? 1 : 0) | (L < K && rq.state == CUT_TIES ? 2 : 0);
        if (sparse) {
            up.n = find_ties(up, uq, (need & 1) | 4, rp, rq, dl);
            up.list = dl.list[t >> 6];
            if (need & 2) {
                const MayKeep<DT> may(rp);
                const float yq = key_value(rq.cut);
                bool hit = false;
                for (int i = 0; i < up.count(); ++i) {
                    const int g = up.group(i);
                    if (may(gp.load(g)))
                        hit |= equal_count<DT>(gq.load(g), yq) != 0;
                }
                need = __syncthreads_or(hit) ? 2 : 0;
            } else {
                need = 0;
            }
        }
        if (need)
            find_ties(up, uq, need, rp, rq, dl);
        __syncthreads();
        const double u = (double)unif[(size_t)b * (K + 1) + K];
        auto draw = [&](auto p, auto q) SV_INLINE {
            // the residual; then, where nothing is left of p - q, p
#pragma nounroll
            for (bool both = L < K;; both = false) {
                id = draw_row(up, MayKeep<DT>(rp), u, dl, ResidualLaw<DT, decltype(p)>{p, q, gq, both});
                if (id >= 0 || !both)
                    break;
                __syncthreads();
            }
        };
        if constexpr (DT == 1)
            draw(TableLaw(rp, V, 1.0 / rp.z, tables[0]), TableLaw(rq, V, 1.0 / rq.z, tables[1]));
        else
            draw(DirectLaw<DT>{uniform(rp), uniform(1.0 / rp.z)}, DirectLaw<DT>{uniform(rq), uniform(1.0 / rq.z)});
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
