// Sampling: temperature, top-k, top-p and min-p over the logits of a decode
// step, without sorting them.
//
// Mathematics.  Tokens are ordered by the 64-bit key (logit descending, index
// ascending), unique per token, so top-k and top-p each keep the keys up to a
// cut.  A cut is found by counting: a histogram over bins that follow the
// order, the bin in which the running count (or weight) reaches its target,
// then the same inside that bin, until few enough candidates are left to rank
// them by comparing each with all.  The first bins are linear in the logit,
// from the largest to the least or 32 octaves of weight down; later ones split
// the bin's range of keys.
//
// Weights 2^-d, d = (max - z) log2(e) / temperature, are 64-bit fixed point
// (2^44 for d = 0), accurate to 2^-30 of themselves or to 2^-44, whichever is
// more (the relative figure holds from 2^-14 on): d is carried as a pair of fp32
// numbers, 2^-d as integers (32-entry table times a polynomial of exp(-a), a <
// ln 2 / 32).  Integer sums do not depend on their order, so neither does the
// token, and the cumulative sums keep the accuracy that a 150,000-token
// vocabulary asks for (fp32 sums would move a boundary by more than a token's
// probability).
//
// Short cut.  Where the candidates up to the bin that holds the cut are at most
// 1024 (any usual top-k; top-p of a peaked distribution), they are gathered in
// one CTA, which does the rest alone: every filter keeps a prefix of the order,
// so ranks and running weights among the candidates decide all three.
//
// Work split.  One cluster of CTAs per row (up to 16: a row of 0.5 MB is
// spread over 16 SMs), each CTA keeping its share of the row in shared
// memory; histograms are joined through distributed shared memory.  What
// bounds it is latency: the row is read once, then cluster barriers follow.
// Measured (one GB300, device time): one row of 128,256 with all filters 12.8
// us (its bytes take 0.08), 16 rows of 151,936 with mixed settings 28.3 us.
#include <cooperative_groups.h>

#include <algorithm>

#include "dev_serve.cuh"

namespace cg = cooperative_groups;

namespace mk {

constexpr int SMP_THREADS = 512, SMP_WARPS = SMP_THREADS / 32;
constexpr int SMP_BINS = 2048;                   // first-level bins
constexpr int SMP_COARSE = 64, SMP_FINE = SMP_BINS / SMP_COARSE;  // first-level bins are searched in two steps
constexpr int SMP_CAP = 1024;                    // candidates ranked directly
constexpr int SMP_MAXCTAS = 16;
constexpr int SMP_CHUNK = 38912;                 // logits per CTA at most (152 KB)
constexpr int SMP_ROW = 128;                     // logits per warp pass
constexpr uint64_t KEY_NONE = ~0ull;

struct SmpParams {
    const void *logits;
    int64_t row_stride;
    int vocab, chunk;
    const float *u;
    int *tokens;
    float *logprob;
    const float *temperature_rows, *top_p_rows, *min_p_rows;
    const int *top_k_rows;
    float temperature, top_p, min_p;
    int top_k;
};

struct alignas(16) SmpShared {  // the logits behind it are read 16 bytes at a time
    uint32_t table[32];                             // 2^31 2^(-i/32)
    unsigned long long best[SMP_MAXCTAS];           // every CTA's largest (ordered logit, index)
    uint32_t least[SMP_MAXCTAS];                    // every CTA's least logit above -inf, ordered
    unsigned long long slice_w[SMP_MAXCTAS];        // every CTA's slice of the histogram
    uint32_t slice_n[SMP_MAXCTAS];
    unsigned long long lo[SMP_MAXCTAS], hi[SMP_MAXCTAS];  // every CTA's least and largest key in the bin
    unsigned long long kept[SMP_MAXCTAS];           // every CTA's kept weight
    unsigned long long before_w, need, total;       // the bin found: weight before it; what was looked for
    uint32_t before_n, bin_n;
    int bin;
    unsigned long long cut, cut_w;                  // the cut found and the weight up to it
    uint32_t cands;
    unsigned long long red[SMP_WARPS];
    uint32_t red_n[SMP_WARPS];
    // sums over all CTAs, added by them (one set for each of two searches), and
    // over the found coarse bin's fine bins
    alignas(16) unsigned long long coarse_w[2][SMP_COARSE];
    unsigned long long fine_w[SMP_FINE];
    uint32_t coarse_n[2][SMP_COARSE], fine_n[SMP_FINE];
    uint32_t hist[4][SMP_BINS];                     // count; weight in 16-bit pieces
    unsigned long long ckey[SMP_CAP], cw[SMP_CAP];  // candidates (in CTA 0)
};

// Keys rise in sampling order: the larger logit first, then the lower index.
DEV uint32_t ordered_bits(float x) {
    const uint32_t b = __float_as_uint(x);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
DEV unsigned long long sample_key(float x, int i) {
    return ((unsigned long long)(~ordered_bits(x)) << 32) | (uint32_t)i;
}

// 2^31 2^(-i/32)
__constant__ uint32_t c_table[32] = {
    2147483648u, 2101467502u, 2056437387u, 2012372174u, 1969251188u, 1927054196u, 1885761398u, 1845353420u,
    1805811301u, 1767116489u, 1729250827u, 1692196547u, 1655936265u, 1620452965u, 1585730000u, 1551751076u,
    1518500250u, 1485961921u, 1454120821u, 1422962010u, 1392470869u, 1362633090u, 1333434672u, 1304861917u,
    1276901417u, 1249540052u, 1222764986u, 1196563654u, 1170923762u, 1145833280u, 1121280436u, 1097253708u};

// floor (up: ceiling) of f x for 0 <= f < 1, exactly: f = mantissa 2^-s.  (FP64
// arithmetic is to be kept out of this file: a few instructions of it in
// every thread cost more than the pass over the logits.)
DEV unsigned long long frac_of(float f, unsigned long long x, bool up) {
    const uint32_t bits = __float_as_uint(f);
    const int s = 150 - (int)(bits >> 23);
    if (s >= 128) return up && bits ? 1 : 0;  // below 2^-102 (or 0)
    const unsigned long long m = (bits & 0x7fffffu) | 0x800000u, hi = __umul64hi(m, x), lo = m * x;
    unsigned long long q, rest;
    if (s < 64) {
        q = hi << (64 - s) | lo >> s;
        rest = lo << (64 - s);
    } else {
        q = s == 64 ? hi : hi >> (s - 64);
        rest = lo | (s == 64 ? 0 : hi << (128 - s));
    }
    return q + (up && rest ? 1 : 0);
}

struct Weigher {
    float top, ch, cl;  // the row's maximum; log2(e) / temperature as a pair of fp32
    const uint32_t *table;
    DEV float octaves(float x) const { return (top - x) * ch; }  // d in fp32: monotone in x
    // 2^44 2^-d, without branches, so that several weights overlap
    DEV unsigned long long operator()(float x) const {
        const float dh = top - x;
        const float bp = dh - top;
        const float dl = (top - (dh - bp)) + (-x - bp);  // dh + dl = top - x exactly
        const float t = fminf(dh * ch, 47.f);            // (NaN too) from 46 on the weight is 0
        const float te = t < 46.f ? fmaf(dh, ch, -t) + fmaf(dh, cl, dl * ch) : 0.f;
        const int n = __float2int_rz(t);
        // d in 32.32 fixed point; t - n is exact, te below 2^-17
        const long long d = max(0ll, ((long long)n << 32) + (long long)__float2uint_rz((t - (float)n) * 4294967296.f) +
                                         (long long)__float2int_rn(te * 4294967296.f));
        const uint32_t f = (uint32_t)d;
        // 2^-f = table x exp(-a), a = (f mod 1/32) ln 2 < 0.0217: terms to a^4 / 24 leave 4e-11
        const uint32_t a = __umulhi(f & 0x07ffffffu, 2977044472u);  // ln 2 in 0.32
        uint32_t q = 715827883u - __umulhi(a, 178956971u);         // 1/6 - a/24
        q = 0x80000000u - __umulhi(a, q);                          // 1/2 - a q
        q = 0xffffffffu - __umulhi(a, q);                          // 1 - a q
        const uint32_t e = 0x80000000u - (__umulhi(a, q) >> 1);    // 1 - a q, in 1.31
        const unsigned long long prod = (unsigned long long)table[f >> 27] * e;  // 2.62
        const unsigned long long r = prod >> min(18 + (int)(d >> 32), 63);
        return x == top ? 1ull << 44 : r;  // (the largest may be infinite)
    }
};

// log(w / total) = -log1p(rest / w): fp32 throughout, a few last places of the
// result also near 0 (the conversions and the quotient half a place each).
DEV float log_share(unsigned long long w, unsigned long long total) {
    return -log1pf(__fdiv_rn(__ull2float_rn(total - w), __ull2float_rn(w)));
}
DEV unsigned long long warp_sum64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    return v;
}
DEV unsigned long long warp_min64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = min(v, __shfl_xor_sync(FULL, v, o));
    return v;
}

// One row per cluster.  Every CTA keeps logits [rank * chunk, ...) in shared
// memory; `x` behind the row's end are -inf.
struct Sampler {
    const SmpParams &p;
    SmpShared &s;
    float *x;
    unsigned long long *rows;  // kept weight of each 128-logit pass
    cg::cluster_group cl;
    int rank, ctas, first, n;  // n: multiple of 128
    Weigher w;
    float bins;  // bins per octave of weight

    DEV float4 four(int i) const { return *reinterpret_cast<const float4 *>(x + i); }

    // The first key position at which the running count reaches `need_n` (by
    // count) or the running weight reaches `need_w`, over keys <= limit, all
    // of which hold `limit`; returns that key, and the weight up to it.
    DEV unsigned long long find(bool by_weight, unsigned long long need, unsigned long long limit,
                                unsigned long long &upto) {
        const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
        unsigned long long lo = 0, hi = limit, w_before = 0;
        uint32_t n_before = 0;
        bool octave = true;  // bins: octaves of weight first, then keys
        int shift = 0;
        while (true) {
            for (int i = tid; i < 4 * SMP_BINS; i += SMP_THREADS) s.hist[0][i] = 0;
            __syncthreads();
            for (int i = tid * 4; i < n; i += SMP_THREADS * 4) {
                const float4 v = four(i);
                const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const unsigned long long key = sample_key(e[j], first + i + j);
                    if (e[j] == -INFINITY || key < lo || key > hi) continue;
                    const int bin = octave ? bin_of(e[j]) : (int)((key - lo) >> shift);
                    const unsigned long long ww = w(e[j]);
                    atomicAdd(&s.hist[0][bin], 1u);
                    atomicAdd(&s.hist[1][bin], (uint32_t)ww & 0xffffu);
                    atomicAdd(&s.hist[2][bin], (uint32_t)(ww >> 16) & 0xffffu);
                    atomicAdd(&s.hist[3][bin], (uint32_t)(ww >> 32));
                }
            }
            cl.sync();
            // this CTA's slice of the bins over all CTAs
            const int per = SMP_BINS / ctas;
            unsigned long long bw = 0;
            uint32_t bn = 0;
            // threads hold consecutive bins of the slice (per <= 2048: up to 4 each)
            constexpr int M = SMP_BINS / SMP_THREADS;
            unsigned long long tw[M];
            uint32_t tn[M];
#pragma unroll
            for (int k = 0; k < M; ++k) {
                tw[k] = 0;
                tn[k] = 0;
                const int i = tid * M + k;
                if (i < per)
                    for (int r = 0; r < ctas; ++r) {
                        const uint32_t *h = cl.map_shared_rank(&s.hist[0][0], r) + rank * per + i;
                        tn[k] += h[0];
                        tw[k] += (unsigned long long)h[SMP_BINS] + ((unsigned long long)h[2 * SMP_BINS] << 16) +
                                 ((unsigned long long)h[3 * SMP_BINS] << 32);
                    }
                bn += tn[k];
                bw += tw[k];
            }
            // exclusive prefix over the block
            unsigned long long pw = bw;
            uint32_t pn = bn;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long a = __shfl_up_sync(FULL, pw, o);
                const uint32_t b = __shfl_up_sync(FULL, pn, o);
                if (lane >= o) {
                    pw += a;
                    pn += b;
                }
            }
            if (lane == 31) {
                s.red[warp] = pw;
                s.red_n[warp] = pn;
            }
            __syncthreads();
            unsigned long long all_w = 0;
            uint32_t all_n = 0;
            unsigned long long my_w = pw - bw;
            uint32_t my_n = pn - bn;
#pragma unroll
            for (int i = 0; i < SMP_WARPS; ++i) {
                if (i < warp) {
                    my_w += s.red[i];
                    my_n += s.red_n[i];
                }
                all_w += s.red[i];
                all_n += s.red_n[i];
            }
            if (tid < ctas) {
                *cl.map_shared_rank(&s.slice_w[rank], tid) = all_w;
                *cl.map_shared_rank(&s.slice_n[rank], tid) = all_n;
            }
            cl.sync();
            unsigned long long sw = w_before;
            uint32_t sn = n_before;
            for (int r = 0; r < rank; ++r) {
                sw += s.slice_w[r];
                sn += s.slice_n[r];
            }
            my_w += sw;
            my_n += sn;
#pragma unroll
            for (int k = 0; k < M; ++k) {
                const bool hit = by_weight ? (my_w < need && my_w + tw[k] >= need) : (my_n < need && my_n + tn[k] >= need);
                if (hit)
                    for (int r = 0; r < ctas; ++r) {
                        SmpShared *o = cl.map_shared_rank(&s, r);
                        o->bin = rank * per + tid * M + k;
                        o->before_w = my_w;
                        o->before_n = my_n;
                        o->bin_n = tn[k];
                    }
                my_w += tw[k];
                my_n += tn[k];
            }
            if (tid == 0) s.cands = 0;
            cl.sync();
            const int bin = s.bin;
            w_before = s.before_w;
            n_before = s.before_n;
            const uint32_t count = s.bin_n;
            // the bin's keys: gathered in CTA 0 if few, else their range for the next level
            unsigned long long mn = KEY_NONE, mx = 0;
            SmpShared *lead = cl.map_shared_rank(&s, 0);
            for (int i = tid * 4; i < n; i += SMP_THREADS * 4) {
                const float4 v = four(i);
                const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const unsigned long long key = sample_key(e[j], first + i + j);
                    if (e[j] == -INFINITY || key < lo || key > hi) continue;
                    if ((octave ? bin_of(e[j]) : (int)((key - lo) >> shift)) != bin) continue;
                    if (count <= SMP_CAP) {
                        const uint32_t at = atomicAdd(&lead->cands, 1u);
                        lead->ckey[at] = key;
                        lead->cw[at] = w(e[j]);
                    } else {
                        mn = min(mn, key);
                        mx = max(mx, key);
                    }
                }
            }
            if (count <= SMP_CAP) break;
            mn = warp_min64(mn);
            mx = ~warp_min64(~mx);
            __syncthreads();  // s.red was read
            if (lane == 0) {
                s.red[warp] = mn;
                s.ckey[warp] = mx;
            }
            __syncthreads();
            if (tid < ctas) {
                for (int i = 0; i < SMP_WARPS; ++i) {
                    mn = min(mn, s.red[i]);
                    mx = max(mx, s.ckey[i]);
                }
                *cl.map_shared_rank(&s.lo[rank], tid) = mn;
                *cl.map_shared_rank(&s.hi[rank], tid) = mx;
            }
            cl.sync();
            lo = KEY_NONE;
            hi = 0;
            for (int r = 0; r < ctas; ++r) {
                lo = min(lo, s.lo[r]);
                hi = max(hi, s.hi[r]);
            }
            octave = false;
            shift = max(0, 64 - __clzll(hi - lo) - 11);
        }
        cl.sync();
        if (rank == 0) {
            const int count = (int)s.bin_n, size = list_size(count);
            sort(count, size);
            announce(by_weight, need, n_before, w_before, count, size);
        }
        cl.sync();
        upto = s.cut_w;
        return s.cut;
    }

    // CTA 0, after sort: the key at which the target is reached, to all CTAs.
    DEV void announce(bool by_weight, unsigned long long need, uint32_t n_before, unsigned long long w_before, int count,
                      int size) const {
        unsigned long long before = w_before + list_before(size);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int i = 2 * (int)threadIdx.x + k;
            if (i >= count) break;
            const unsigned long long with = before + s.cw[i];
            if (by_weight ? before < need && with >= need : n_before + i + 1 == need)
                for (int r = 0; r < ctas; ++r) {
                    SmpShared *o = cl.map_shared_rank(&s, r);
                    o->cut = s.ckey[i];
                    o->cut_w = with;
                }
            before = with;
        }
    }

    // First-level histogram of every logit above -inf, joined over the cluster.
    // Finds the bin in which the running count (by_weight: weight) reaches its
    // target: `need` of the count, or the fraction `share` of the weight.
    // s.bin (-1: there are fewer than `need`), s.before_n / before_w, s.bin_n,
    // and the total weight are the same in every CTA afterwards.
    DEV void first_bin(int set, bool by_weight, uint32_t need_n, float share, unsigned long long &need, unsigned long long &total) {
        const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
        for (int i = tid; i < (by_weight ? 4 : 1) * SMP_BINS; i += SMP_THREADS) s.hist[0][i] = 0;
        if (tid == 0) s.cands = 0;  // before any CTA's gather: a cluster barrier comes first
        if (tid < SMP_FINE) s.fine_n[tid] = 0, s.fine_w[tid] = 0;
        __syncthreads();
        for (int i = tid * 4; i < n; i += SMP_THREADS * 4) {
            const float4 v = four(i);
            const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (e[j] == -INFINITY) continue;
                const int bin = bin_of(e[j]);
                atomicAdd(&s.hist[0][bin], 1u);
                if (by_weight) {
                    const unsigned long long ww = w(e[j]);
                    atomicAdd(&s.hist[1][bin], (uint32_t)ww & 0xffffu);
                    atomicAdd(&s.hist[2][bin], (uint32_t)(ww >> 16) & 0xffffu);
                    atomicAdd(&s.hist[3][bin], (uint32_t)(ww >> 32));
                }
            }
        }
        __syncthreads();
        {   // coarse sums to every CTA: 8 threads a coarse bin
            constexpr int T = SMP_THREADS / SMP_COARSE, M = SMP_FINE / T;
            const int c = tid / T;
            uint32_t cn = 0;
            unsigned long long cw = 0;
#pragma unroll
            for (int k = 0; k < M; ++k) {
                const int i = c * SMP_FINE + tid % T * M + k;
                cn += s.hist[0][i];
                if (by_weight) cw += hist_weight(&s.hist[0][i]);
            }
#pragma unroll
            for (int o = 1; o < T; o <<= 1) {
                cn += __shfl_xor_sync(FULL, cn, o);
                cw += __shfl_xor_sync(FULL, cw, o);
            }
            for (int r = tid % T; r < ctas; r += T) {
                SmpShared *q = cl.map_shared_rank(&s, r);
                atomicAdd(&q->coarse_n[set][c], cn);
                if (by_weight) atomicAdd(&q->coarse_w[set][c], cw);
            }
        }
        cl.sync();
        if (warp == 0) {  // lane: coarse bins 2 lane, 2 lane + 1
            const uint32_t cn[2] = {s.coarse_n[set][2 * lane], s.coarse_n[set][2 * lane + 1]};
            const unsigned long long cw[2] = {s.coarse_w[set][2 * lane], s.coarse_w[set][2 * lane + 1]};
            uint32_t pn = cn[0] + cn[1];
            unsigned long long pw = cw[0] + cw[1];
            running(lane, pn, pw);
            const unsigned long long all = __shfl_sync(FULL, pw, 31);
            const unsigned long long goal = by_weight ? max(frac_of(fmaxf(share, 0.f), all, true), 1ull) : need_n;
            if (lane == 0) {
                s.bin = -1;
                s.need = goal;
                s.total = all;
            }
            __syncwarp();
            unsigned long long bw = pw - cw[0] - cw[1];
            uint32_t bn = pn - cn[0] - cn[1];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (by_weight ? bw < goal && bw + cw[k] >= goal : bn < goal && bn + cn[k] >= goal) {
                    s.bin = 2 * lane + k;
                    s.before_w = bw;
                    s.before_n = bn;
                }
                bw += cw[k];
                bn += cn[k];
            }
        }
        __syncthreads();
        need = s.need;
        total = s.total;
        const int c = s.bin;
        if (c >= 0) {
            if (warp < ctas) {
                const uint32_t *h = cl.map_shared_rank(&s.hist[0][c * SMP_FINE + lane], warp);
                atomicAdd(&s.fine_n[lane], h[0]);
                if (by_weight) atomicAdd(&s.fine_w[lane], hist_weight(h));
            }
            __syncthreads();
            if (warp == 0) {
                const uint32_t fn = s.fine_n[lane];
                const unsigned long long fw = s.fine_w[lane];
                uint32_t pn = fn;
                unsigned long long pw = fw;
                running(lane, pn, pw);
                const unsigned long long bw = s.before_w + pw - fw;
                const uint32_t bn = s.before_n + pn - fn;
                __syncwarp();
                if (by_weight ? bw < need && bw + fw >= need : bn < need && bn + fn >= need) {
                    s.bin = c * SMP_FINE + lane;
                    s.before_w = bw;
                    s.before_n = bn;
                    s.bin_n = fn;
                }
            }
            __syncthreads();
        }
    }
    DEV static unsigned long long hist_weight(const uint32_t *h) {
        return (unsigned long long)h[SMP_BINS] + ((unsigned long long)h[2 * SMP_BINS] << 16) +
               ((unsigned long long)h[3 * SMP_BINS] << 32);
    }
    // inclusive sums over the warp
    DEV static void running(int lane, uint32_t &pn, unsigned long long &pw) {
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t a = __shfl_up_sync(FULL, pn, o);
            const unsigned long long b = __shfl_up_sync(FULL, pw, o);
            if (lane >= o) {
                pn += a;
                pw += b;
            }
        }
    }

    // Logits of bins lo .. hi into CTA 0's list (ends with a cluster barrier).
    DEV void gather(int lo, int hi) {
        SmpShared *lead = cl.map_shared_rank(&s, 0);
        for (int i = threadIdx.x * 4; i < n; i += SMP_THREADS * 4) {
            const float4 v = four(i);
            const float e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (e[j] == -INFINITY) continue;
                const int bin = bin_of(e[j]);
                if (bin < lo || bin > hi) continue;
                const uint32_t at = atomicAdd(&lead->cands, 1u);
                lead->ckey[at] = sample_key(e[j], first + i + j);
                lead->cw[at] = w(e[j]);
            }
        }
        cl.sync();
    }

    // Sorts the list's `count` candidates by key, all threads; the entries up
    // to `size`, a power of two, are filled with KEY_NONE, weight 0.  Up to 256
    // by counting, for each, the smaller ones (2.5 us for two sorts of 100, a
    // step of the bitonic form costs 0.09 us); above, the comparisons'
    // shared-memory reads would take longer than the bitonic steps.
    DEV void sort(int count, int size) const {
        const int tid = threadIdx.x;
        if (size <= 256) {
            const int lg = min(5, 32 - __clz(SMP_THREADS / size) - 1), g = 1 << lg, i = tid >> lg;
            const unsigned long long key = i < count ? s.ckey[i] : KEY_NONE, w = i < count ? s.cw[i] : 0;
            uint32_t place = 0;
            if (i < count) {
#pragma unroll 4
                for (int j = tid & (g - 1); j < count; j += g) place += s.ckey[j] < key;
            }
            for (int o = 1; o < g; o <<= 1) place += __shfl_xor_sync(FULL, place, o);
            __syncthreads();
            if ((tid & (g - 1)) == 0 && i < size) {
                s.ckey[i < count ? place : i] = key;
                s.cw[i < count ? place : i] = w;
            }
            __syncthreads();
            return;
        }
        for (int i = count + tid; i < size; i += SMP_THREADS) {
            s.ckey[i] = KEY_NONE;
            s.cw[i] = 0;
        }
        __syncthreads();
        for (int run = 2; run <= size; run *= 2)
            for (int step = run / 2; step > 0; step /= 2) {
                if (tid < size / 2) {
                    const int i = 2 * tid - (tid & (step - 1)), j = i + step;
                    const unsigned long long a = s.ckey[i], b = s.ckey[j];
                    if ((a > b) == ((i & run) == 0)) {
                        const unsigned long long wa = s.cw[i], wb = s.cw[j];
                        s.ckey[i] = b;
                        s.ckey[j] = a;
                        s.cw[i] = wb;
                        s.cw[j] = wa;
                    }
                }
                __syncthreads();
            }
    }
    // This thread's candidates are 2 tid and 2 tid + 1: the weight before them,
    // in the list's order.
    DEV unsigned long long list_before(int size) const {
        const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
        const unsigned long long own = 2 * tid < size ? s.cw[2 * tid] + s.cw[2 * tid + 1] : 0;
        uint32_t none = 0;
        unsigned long long sum = own;
        running(lane, none, sum);
        __syncthreads();  // s.red was read
        if (lane == 31) s.red[warp] = sum;
        __syncthreads();
        sum -= own;
#pragma unroll
        for (int i = 0; i < SMP_WARPS; ++i)
            if (i < warp) sum += s.red[i];
        return sum;
    }
    DEV static int list_size(int count) { return count <= 2 ? 2 : 1 << (32 - __clz(count - 1)); }

    DEV int bin_of(float v) const { return (int)fminf((float)(SMP_BINS - 1), w.octaves(v) * bins); }
};

// The rest of a row among the candidates of CTA 0's list, which hold every
// logit up to the cuts: top_k of them (or all), then top-p (`need` of the
// weight if it is known, else top_p of the top_k's), then those >= least.
static __device__ __noinline__ void finish_few(const Sampler &k, int count, int top_k, float top_p, unsigned long long need,
                                               float least, unsigned long long least_w, float u, int *token, float *logprob) {
    SmpShared &s = k.s;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int size = k.list_size(count);
    k.sort(count, size);  // rank = place in the list
    unsigned long long before = k.list_before(size);
    const int i0 = 2 * tid;
    if (i0 < count) {
        const unsigned long long w0 = s.cw[i0];
        if (i0 == top_k - 1) s.cut_w = before + w0;
        if (i0 + 1 == top_k - 1) s.cut_w = before + w0 + s.cw[i0 + 1];
    }
    __syncthreads();
    if (need == 0) {
        need = s.cut_w;
        if (top_p < 1.f) need = max(frac_of(fmaxf(top_p, 0.f), s.cut_w, true), 1ull);
    }
    // what is dropped goes to the end of the list, without weight; the rest in the vocabulary's order
    unsigned long long sum = 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = i0 + j;
        if (i >= count) break;
        const unsigned long long key = s.ckey[i], w = s.cw[i];
        const uint32_t ob = ~(uint32_t)(key >> 32);
        const float z = __uint_as_float(ob & 0x80000000u ? ob & 0x7fffffffu : ~ob);
        const bool keep = i < top_k && before < need && z >= least && w >= least_w;
        before += w;
        sum += keep ? w : 0;
        s.ckey[i] = keep ? (unsigned long long)(uint32_t)key : KEY_NONE;
        s.cw[i] = keep ? w : 0;
    }
    const int kept = __syncthreads_count(i0 < count && s.ckey[i0] != KEY_NONE) + __syncthreads_count(i0 + 1 < count && s.ckey[i0 + 1] != KEY_NONE);
    sum = warp_sum64(sum);
    if (lane == 0) s.red[warp] = sum;
    __syncthreads();
    unsigned long long total = 0;
    for (int i = 0; i < SMP_WARPS; ++i) total += s.red[i];
    // a prefix of the list was kept: the rest holds no weight and need not be sorted
    const int ksize = k.list_size(kept);
    k.sort(kept, ksize);
    const unsigned long long target = frac_of(u, total, false);
    before = k.list_before(ksize);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int i = i0 + j;
        if (i >= kept) break;
        const unsigned long long w = s.cw[i];
        if (before <= target && target < before + w) {
            *token = (int)(uint32_t)s.ckey[i];
            if (logprob) *logprob = log_share(w, total);
        }
        before += w;
    }
}

template <bool BF16>
__global__ void __launch_bounds__(SMP_THREADS, 2) sample_kernel(const SmpParams p) {
    SmpShared &s = *reinterpret_cast<SmpShared *>(mk_smem);
    float *x = reinterpret_cast<float *>(mk_smem + sizeof(SmpShared));
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), ctas = (int)cl.num_blocks();
    const int row = blockIdx.x / ctas, tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int first = rank * p.chunk, have = min(p.chunk, p.vocab - first), n = p.chunk;
    unsigned long long *rows = reinterpret_cast<unsigned long long *>(x + p.chunk);

    // the row's share into shared memory, and its largest (logit, index)
    float top = -INFINITY, bottom = INFINITY;
    int at = 0;
    const auto put = [&](int i, float v) {
        v = v != v ? -INFINITY : v + 0.f;  // -0 counts as 0
        x[i] = v;
        if (v > -INFINITY) bottom = fminf(bottom, v);
        if (v > top || (v == top && first + i < at)) {
            top = v;
            at = first + i;
        }
    };
    constexpr int VEC = BF16 ? 8 : 4;
    const char *src = static_cast<const char *>(p.logits) + (row * p.row_stride + first) * (BF16 ? 2 : 4);
    const int vecs = have > 0 && (uintptr_t)src % 16 == 0 ? have / VEC : 0;
#pragma unroll 4
    for (int i = tid; i < vecs; i += SMP_THREADS) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(src) + i);
        const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if constexpr (BF16) {
                put(8 * i + 2 * j, __uint_as_float(e[j] << 16));
                put(8 * i + 2 * j + 1, __uint_as_float(e[j] & 0xffff0000u));
            } else {
                put(4 * i + j, __uint_as_float(e[j]));
            }
        }
    }
    for (int i = vecs * VEC + tid; i < n; i += SMP_THREADS) {
        float v = -INFINITY;
        if (i < have)
            v = BF16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(src)[i] << 16)
                     : reinterpret_cast<const float *>(src)[i];
        put(i, v);
    }
    // largest (ordered logit, ~index) of the block, then of the cluster
    unsigned long long best = ((unsigned long long)ordered_bits(top) << 32) | (uint32_t)~at;
    best = ~warp_min64(~best);
    const uint32_t low = __reduce_min_sync(FULL, ordered_bits(bottom));
    if (lane == 0) {
        s.red[warp] = best;
        s.red_n[warp] = low;
    }
    if (tid < 32) s.table[tid] = c_table[tid];
    if (tid < 2 * SMP_COARSE) s.coarse_n[0][tid] = 0, s.coarse_w[0][tid] = 0;  // before the cluster barrier
    __syncthreads();
    if (tid < ctas) {
        uint32_t lo = ~0u;
        for (int i = 0; i < SMP_WARPS; ++i) {
            best = max(best, s.red[i]);
            lo = min(lo, s.red_n[i]);
        }
        *cl.map_shared_rank(&s.best[rank], tid) = best;
        *cl.map_shared_rank(&s.least[rank], tid) = lo;
    }
    cl.sync();
    best = 0;
    uint32_t lob = ~0u;
#pragma unroll
    for (int r = 0; r < SMP_MAXCTAS; ++r)
        if (r < ctas) {
            best = max(best, s.best[r]);
            lob = min(lob, s.least[r]);
        }
    const int arg = (int)~(uint32_t)best;
    const uint32_t ob = (uint32_t)(best >> 32);
    top = __uint_as_float(ob & 0x80000000u ? ob & 0x7fffffffu : ~ob);

    const float temp = p.temperature_rows ? p.temperature_rows[row] : p.temperature;
    const int top_k = p.top_k_rows ? p.top_k_rows[row] : p.top_k;
    const float top_p = p.top_p_rows ? p.top_p_rows[row] : p.top_p;
    const float min_p = p.min_p_rows ? p.min_p_rows[row] : p.min_p;
    if (!(temp > 0.f) || top_k == 1 || top == -INFINITY) {  // the same in the whole cluster
        if (rank == 0 && tid == 0) {
            p.tokens[row] = top == -INFINITY ? 0 : arg;
            if (p.logprob) p.logprob[row] = top == -INFINITY ? -INFINITY : 0.f;
        }
        return;
    }
    // log2(e) / temperature as ch + cl: quotient, then the exact remainder's
    const float log2e = 1.44269502f, log2e_lo = 1.92596303e-8f, ch = __fdiv_rn(log2e, temp);
    const float cl_ = ch < INFINITY ? (fmaf(-ch, temp, log2e) + log2e_lo) / temp : 0.f;
    Sampler k{p, s, x, rows, cl, rank, ctas, first, n, {top, ch, cl_, s.table}, 0.f};
    // the logits' span in octaves, 32 at most; all in one bin if they are equal
    const float span = fminf(k.w.octaves(__uint_as_float(lob & 0x80000000u ? lob & 0x7fffffffu : ~lob)), 32.f);
    k.bins = span > 0.f ? (float)SMP_BINS / span : 0.f;

    const float u = fminf(fmaxf(p.u[row], 0.f), 0x1.fffffep-1f);
    // min_p as a least weight; from 1 on only the largest logit itself
    const float least = min_p >= 1.f ? top : -INFINITY;
    const unsigned long long least_w = min_p > 0.f && min_p < 1.f ? frac_of(min_p, 1ull << 44, true) : 0;
    unsigned long long cut = sample_key(-3.402823466e38f, 0x7fffffff), cut_w = 0;  // every finite logit
    bool by_k = top_k > 0 && top_k < p.vocab, by_p = top_p < 1.f;
    if (by_k || by_p) {
        unsigned long long need, all;
        k.first_bin(0, !by_k, top_k, top_p, need, all);
        if (by_k && s.bin < 0) {  // fewer than top_k logits above -inf: no cut there
            by_k = false;
            cl.sync();  // the bins were read
            if (by_p) k.first_bin(1, true, 0, top_p, need, all);
        }
        const int bin = s.bin;
        const uint32_t upto = s.before_n + s.bin_n;
        if ((by_k || by_p) && upto <= SMP_CAP) {
            k.gather(0, bin);
            if (rank != 0) return;
            finish_few(k, upto, by_k ? top_k : (int)upto, by_p ? top_p : 1.f, by_p && !by_k ? need : 0, least, least_w, u,
                       p.tokens + row, p.logprob ? p.logprob + row : nullptr);
            return;
        }
        if (by_k) {
            cl.sync();  // the bins were read
            cut = k.find(false, top_k, cut, cut_w);
            if (by_p) {
                need = max(frac_of(fmaxf(top_p, 0.f), cut_w, true), 1ull);
                cut = k.find(true, need, cut, cut_w);
            }
        } else if (by_p && s.bin_n <= SMP_CAP) {
            const uint32_t count = s.bin_n;
            const unsigned long long before = s.before_w;
            k.gather(bin, bin);
            if (rank == 0) {
                const int size = k.list_size((int)count);
                k.sort((int)count, size);
                k.announce(true, need, 0, before, (int)count, size);
            }
            cl.sync();
            cut = s.cut;
        } else if (by_p) {
            cl.sync();  // the bins were read
            cut = k.find(true, need, cut, cut_w);
        }
    }
    // weight of what a pass keeps: per 128 logits (rows), per CTA, per cluster
    const auto kept = [&](float v, int i) -> unsigned long long {
        const unsigned long long ww = k.w(v);
        return v >= least && sample_key(v, first + i) <= cut && ww >= least_w ? ww : 0;
    };
    const auto kept_weight = [&]() {
        for (int r = warp; r < n / SMP_ROW; r += SMP_WARPS) {
            const int i = r * SMP_ROW + lane * 4;
            const float4 v = k.four(i);
            unsigned long long sum = kept(v.x, i) + kept(v.y, i + 1) + kept(v.z, i + 2) + kept(v.w, i + 3);
            sum = warp_sum64(sum);
            if (lane == 0) rows[r] = sum;
        }
        __syncthreads();
        unsigned long long sum = 0;
        for (int r = tid; r < n / SMP_ROW; r += SMP_THREADS) sum += rows[r];
        sum = warp_sum64(sum);
        if (lane == 0) s.red[warp] = sum;
        __syncthreads();
        if (tid < ctas) {
            unsigned long long a = 0;
            for (int i = 0; i < SMP_WARPS; ++i) a += s.red[i];
            *cl.map_shared_rank(&s.kept[rank], tid) = a;
        }
        cl.sync();
        unsigned long long all = 0;
        for (int r = 0; r < ctas; ++r) all += s.kept[r];
        return all;
    };
    const unsigned long long total = kept_weight();
    const unsigned long long target = frac_of(u, total, false);
    unsigned long long before = 0;
    for (int r = 0; r < rank; ++r) before += s.kept[r];
    if (warp == 0 && before <= target && target < before + s.kept[rank]) {
        // the pass, then the lane, then the logit in which the running sum passes the target
        int r = 0;
        for (int r0 = 0; r0 < n / SMP_ROW; r0 += 32) {
            unsigned long long v = r0 + lane < n / SMP_ROW ? rows[r0 + lane] : 0, q = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned long long a = __shfl_up_sync(FULL, q, o);
                if (lane >= o) q += a;
            }
            const unsigned hit = __ballot_sync(FULL, before + q > target);
            if (hit) {
                const int j = __ffs(hit) - 1;
                r = r0 + j;
                before += __shfl_sync(FULL, q, j) - __shfl_sync(FULL, v, j);
                break;
            }
            before += __shfl_sync(FULL, q, 31);
        }
        const int i = r * SMP_ROW + lane * 4;
        const float4 v = k.four(i);
        const float e[4] = {v.x, v.y, v.z, v.w};
        unsigned long long ww[4], sum = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            ww[j] = kept(e[j], i + j);
            sum += ww[j];
        }
        unsigned long long q = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long a = __shfl_up_sync(FULL, q, o);
            if (lane >= o) q += a;
        }
        before += q - sum;
        if (before <= target && target < before + sum) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (before <= target && target < before + ww[j]) {
                    p.tokens[row] = first + i + j;
                    if (p.logprob) p.logprob[row] = log_share(ww[j], total);
                }
                before += ww[j];
            }
        }
    }
}

}  // namespace mk

using namespace mk;

extern "C" int mk_sample(const mk_sample_desc *d, void *stream) {
    if (!d) return set_error(MK_ERR_INVALID, "null descriptor");
    if (d->batch < 0 || d->vocab <= 0 || (d->batch > 1 && d->row_stride < d->vocab))
        return set_error(MK_ERR_INVALID, "batch negative, vocab not positive, or rows overlap");
    if (d->vocab > SMP_MAXCTAS * SMP_CHUNK) return set_error(MK_ERR_UNSUPPORTED, "vocab above 622592");
    if (d->batch == 0) return MK_OK;
    if (!d->logits || !d->u || !d->tokens) return set_error(MK_ERR_INVALID, "null argument");
    if (d->logits % (d->bf16 ? 2 : 4) || (d->u | d->tokens | d->logprob) % 4)
        return set_error(MK_ERR_INVALID, "a pointer is not aligned to its type");
    // CTAs per row.  Few rows: as many SMs as a cluster may span (one row of
    // 151,936: 14 us with 16, 16 with 8, 22 with 4; its top-p alone 24, 34, 56);
    // many: fewer, longer shares, since clusters of 16 do not pack (32 rows: 23
    // us with 4, 39 with 16 and with 8; 128 rows: 83, 122, 119).  At least what
    // a share of shared memory asks for, at most one per 1024 logits.
    int ctas = d->batch <= 16 ? 16 : 4;
    while (ctas < SMP_MAXCTAS && (d->vocab + ctas - 1) / ctas > SMP_CHUNK) ctas *= 2;
    while (ctas > 1 && d->vocab < ctas * 1024) ctas /= 2;
    if (d->batch > INT32_MAX / SMP_MAXCTAS) return set_error(MK_ERR_UNSUPPORTED, "too many rows");
    SmpParams p{};
    p.logits = reinterpret_cast<const void *>(d->logits);
    p.row_stride = d->row_stride;
    p.vocab = d->vocab;
    p.chunk = ((d->vocab + ctas - 1) / ctas + SMP_ROW - 1) / SMP_ROW * SMP_ROW;
    p.u = reinterpret_cast<const float *>(d->u);
    p.tokens = reinterpret_cast<int *>(d->tokens);
    p.logprob = reinterpret_cast<float *>(d->logprob);
    p.temperature_rows = reinterpret_cast<const float *>(d->temperature_rows);
    p.top_k_rows = reinterpret_cast<const int *>(d->top_k_rows);
    p.top_p_rows = reinterpret_cast<const float *>(d->top_p_rows);
    p.min_p_rows = reinterpret_cast<const float *>(d->min_p_rows);
    p.temperature = d->temperature;
    p.top_k = d->top_k;
    p.top_p = d->top_p;
    p.min_p = d->min_p;
    const int smem = (int)sizeof(SmpShared) + p.chunk * 4 + p.chunk / SMP_ROW * 8;
    void (*f)(const SmpParams) = d->bf16 ? sample_kernel<true> : sample_kernel<false>;
    static std::atomic<uint32_t> ready[SERVE_MAX_DEVICES];
    if (int rc = serve_prepare(reinterpret_cast<const void *>(f), ready, d->bf16 ? 1 : 0, true)) return rc;
    cudaError_t e;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(d->batch * ctas));
    cfg.blockDim = dim3(SMP_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, f, (const SmpParams)p);
    return e == cudaSuccess ? MK_OK : serve_cuda_fail(e, "sampling launch");
}
