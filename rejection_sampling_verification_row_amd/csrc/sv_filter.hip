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
    r.ok = q.ok && !bad && mx > KEY_NEG_INF;
    r.max = key_value(mx);
    r.c = q.c;
    r.cut = KEY_NEG_INF;                            // no key lies below it: all ids
    r.tie = V;
    r.z = 0.0;
    if (!r.ok)
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

// First id, ascending, whose inclusive prefix sum of w(id) exceeds u times the row's sum; the
// last id of positive weight if rounding leaves none.  Returns -1 (and sum 0) for an empty row.
struct DrawLds {
    double wave[FWAVES];
    int found, last;
};

template <typename W>
__device__ int inverse_cdf(int V, double u, double total, DrawLds &lds, W w)
{
    const int t = threadIdx.x, lane = t & 63, wv = t >> 6;
    if (t == 0) {
        lds.found = 0x7fffffff;
        lds.last = -1;
    }
    const double goal = u * total;
    double base = 0.0;
    for (int i0 = 0; i0 < V; i0 += FWG) {
        const int i = i0 + t;
        const double x = i < V ? w(i) : 0.0;
        const double inc = wave_incl_scan(x);
        __syncthreads();
        if (lane == 63)
            lds.wave[wv] = inc;
        __syncthreads();
        double before = base;
        for (int k = 0; k < wv; ++k)
            before += lds.wave[k];
        if (x > 0.0) {
            atomicMax(&lds.last, i);
            if (before + inc > goal)
                atomicMin(&lds.found, i);
        }
        for (int k = 0; k < FWAVES; ++k)
            base += lds.wave[k];
        __syncthreads();
        if (lds.found != 0x7fffffff)
            break;
    }
    return lds.found != 0x7fffffff ? lds.found : lds.last;
}

template <int DT>
__global__ __launch_bounds__(FWG) void k_filter_sample(const char *logits, int V, int64_t stride,
                                                       FilterPtrs f, const float *unif, int *tok,
                                                       float *prob)
{
    __shared__ RedLds red;
    __shared__ DrawLds dl;
    const int n = blockIdx.x;
    const char *row = logits + (size_t)n * stride * Elt<DT>::BYTES;
    const Params q = load_params(f, n, V);
    const RowCut r = cut_by_bisection<DT>(row, V, q, red);
    int id = -1;
    if (r.ok) {
        id = inverse_cdf(V, (double)unif[n], r.z, dl, [&](int i) {
            const float x = Elt<DT>::one(row, i);
            return kept(order_key(x), i, r) ? weight(x, r.max, r.c) : 0.0;
        });
    }
    if (threadIdx.x == 0) {
        tok[n] = id;
        if (prob)
            prob[n] = id < 0 ? NAN : (float)(weight(Elt<DT>::one(row, id), r.max, r.c) / r.z);
    }
}

// Rows of a verify: the B (K+1) target rows, then the B K draft rows.
template <int DT>
__global__ __launch_bounds__(FWG) void k_filter_rows(const char *tgt, const char *drf, int B, int K,
                                                     int V, FilterPtrs ft, FilterPtrs fd,
                                                     RowCut *cuts)
{
    __shared__ RedLds red;
    const int n = blockIdx.x, nt = B * (K + 1);
    const bool is_t = n < nt;
    const char *row = (is_t ? tgt + (size_t)n * V * Elt<DT>::BYTES
                            : drf + (size_t)(n - nt) * V * Elt<DT>::BYTES);
    const Params q = is_t ? load_params(ft, n / (K + 1), V) : load_params(fd, (n - nt) / K, V);
    const RowCut r = cut_by_bisection<DT>(row, V, q, red);
    if (threadIdx.x == 0)
        cuts[n] = r;
}

template <int DT>
__device__ inline double law(const char *row, int id, const RowCut &r)
{
    const float x = Elt<DT>::one(row, id);
    return kept(order_key(x), id, r) ? weight(x, r.max, r.c) / r.z : 0.0;
}

template <int DT>
__global__ __launch_bounds__(FWG) void k_filter_verify(const char *tgt, const char *drf, int B,
                                                       int K, int V, const int *tokens,
                                                       const float *unif, const RowCut *cuts,
                                                       int *acc, int *out, float *probs)
{
    __shared__ RedLds red;
    __shared__ DrawLds dl;
    __shared__ int sL;
    const int b = blockIdx.x, t = threadIdx.x;
    const RowCut *ct = cuts + (size_t)b * (K + 1), *cd = cuts + (size_t)B * (K + 1) + (size_t)b * K;
    const char *trow = tgt + (size_t)b * (K + 1) * V * Elt<DT>::BYTES;
    const char *drow = drf + (size_t)b * K * V * Elt<DT>::BYTES;
    const size_t rb = (size_t)V * Elt<DT>::BYTES;
    if (t < 64) {
        // lane j: position j
        bool ok = t <= K ? ct[t].ok != 0 : true;
        bool take = false;
        double P = 0.0, Q = 0.0;
        if (t < K) {
            const int x = tokens[(size_t)b * K + t];
            ok = ok && cd[t].ok && x >= 0 && x < V;
            if (ok) {
                P = law<DT>(trow + t * rb, x, ct[t]);
                Q = law<DT>(drow + t * rb, x, cd[t]);
                take = P > 0.0 && (double)unif[(size_t)b * (K + 1) + t] * Q <= P;
            }
        }
        const bool good = __ballot(!ok) == 0;
        const unsigned long long rej = __ballot(t < K && !take);
        if (t < K && probs) {
            probs[((size_t)b * K + t) * 2] = good ? (float)P : NAN;
            probs[((size_t)b * K + t) * 2 + 1] = good ? (float)Q : NAN;
        }
        if (t == 0)
            sL = !good ? -1 : rej ? __ffsll(rej) - 1 : K;
    }
    __syncthreads();
    const int L = sL;
    int id = -1;
    if (L >= 0) {
        const char *pr = trow + L * rb, *qr = drow + L * rb;
        const RowCut rp = ct[L];
        double total = rp.z;
        const double u = (double)unif[(size_t)b * (K + 1) + K];
        bool residual = false;
        if (L < K) {
            const RowCut rq = cd[L];
            auto w = [&](int i) { return fmax(law<DT>(pr, i, rp) - law<DT>(qr, i, rq), 0.0); };
            double s = 0.0;
            for (int i = t; i < V; i += FWG)
                s += w(i);
            total = block_sum(s, red.d);
            residual = total > 0.0;
            if (residual)
                id = inverse_cdf(V, u, total, dl, w);
        }
        if (!residual)
            id = inverse_cdf(V, u, L < K ? 1.0 : 1.0, dl, [&](int i) { return law<DT>(pr, i, rp); });
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
        SV_LAUNCH(ln, KIND_TAIL, k_filter_sample<1>, dim3(N), dim3(FWG), 0, x, V, stride, f, unif,
                  tok, prob);
    else
        SV_LAUNCH(ln, KIND_TAIL, k_filter_sample<0>, dim3(N), dim3(FWG), 0, x, V, stride, f, unif,
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
    SV_LAUNCH(ln, KIND_STATS, k_filter_rows<DT>, dim3((unsigned)B * (2 * K + 1)), dim3(FWG), 0, t,
              d, B, K, V, ft, fd, cuts);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess)
        return e;
    SV_LAUNCH(ln, KIND_TAIL, k_filter_verify<DT>, dim3(B), dim3(FWG), 0, t, d, B, K, V, tokens,
              unif, cuts, acc, out, probs);
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
