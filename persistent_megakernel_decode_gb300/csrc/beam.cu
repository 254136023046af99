// Beam search's selection: the best continuations over beams and vocabulary.
//
// Mathematics.  A candidate (beam w, token v) has the total s_w + z_wv -
// log sum_v exp z_wv; the `num` largest of a prompt's beams are wanted, ties to
// the lowest w V + v.  Within a beam the order is that of the logits, so each
// part of a beam's row gives its `num` largest logits and a sum of exponentials;
// the parts' short lists are then ordered by their totals.
//
// The order between beams hangs on the sums: two totals closer than their
// errors would change places.  Totals are therefore formed in 64 bits, and the
// sum is kept to 2^-27 of itself whatever the logits are: equal ones have equal
// errors, which add up (rows of few values, masked tails, bf16), so no error may
// be left to averages.  A part's largest logits are weighed by the fixed-point
// weights of dev_weigh.cuh (2^-30).  The rest are fp32 w (1 + r), w a power of
// 2^(1/32) from a table and r the rest of it from a polynomial: log2(e) in two
// parts for the argument (Cody and Waite's reduction), a table with a short
// polynomial (Tang's exponential).  What a product and a polynomial round away
// is then 2^-24 of r, 2^-6.5 or less; the w are added with what each addition
// loses (Dekker's sum of two).  In all 2^-28.6 a term, and 2^-28.7 for the chain
// of eight small parts.  Partial sums are joined as integers, so no order of
// arrival changes anything.  (With the hardware's 2^f, off by up to 2^-22, the
// sum of a flat row was off by 2^-22.6 and of a normal one by 2^-26, and 16 x 8
// beams took 29.7 us where they take 38.2.)
//
// The largest without sorting: a bound that at least `num` threads' largest
// values reach is found by bisection, one barrier and vote a step; the few
// logits that reach it (at most as many per thread as it holds) are listed.
// Later pieces of the part list what is above the bound; when the list is full
// the bound rises to what the listed allow, and the list shrinks to it (doing so
// now and then, before, cost more than it saved: 31.6 us where 29.1 do).  At the
// end the list is ranked by comparing each with all; where very many are equal it
// is cut by bisection first, here and in the second launch (4 equal flat rows of
// 151,936 logits, 128 continuations: 0.45 ms, with comparisons alone 36).
//
// Work split.  A CTA streams a part of a row, 4096 logits at a time in
// registers, the next piece's loads in flight.  A second, dependent launch orders
// a prompt's candidates, one CTA each.  Each logit is read once, so bytes bound
// it from below; 64 x 8 beams of 151,936 logits take 80 us, 3.5 TB/s, and 16 x 8
// 38, of which the bytes are 10: 28 instructions a logit, half of them its term's
// (as instructions on register pairs throughout 40.6 us; with the next piece's
// loads behind the terms 42), and with the bisection and the rank of each part's
// list 33; the barriers of these; the ramp of two launches.  Three
// CTAs an SM in one wave are the best split (with six, and a cheaper sum, 36 us
// where three took 29; one cluster a row, in registers, 52-99).
#include <algorithm>
#include <climits>

#include "dev_weigh.cuh"

namespace mk {

constexpr int BM_THREADS = 256, BM_WARPS = BM_THREADS / 32;
constexpr int BM_PER = 16, BM_PIECE = BM_THREADS * BM_PER;  // logits per thread and CTA at a time
constexpr int BM_MAXVOCAB = 622592;
constexpr int BM_MAXBEAMS = 64, BM_MAXNUM = 128;
constexpr int BM_CANDIDATES = 8192;                          // of a prompt at most: beams x parts x num
constexpr int BM_MERGE_THREADS = 512;
constexpr int BM_MAXSMS = 256;                               // that parts are planned for

// What the second launch needs of a part beside its list.
struct BeamPart {
    float top;              // the largest logit
    int ref;                // `rest` is in units of 2^(ref - 44)
    unsigned long long list, rest;  // sums: of the listed weights relative to the largest, in 2^-44; of the others
};

struct BeamParams {
    const void *logits;
    int64_t row_stride;
    int vocab, beams, num, chunk, parts, limit, cap;
    const float *scores;
    const uint8_t *finished;
    int end;
    BeamPart *rows;             // workspace: [batch x beams][parts]
    unsigned long long *keys;   // workspace: [batch x beams][parts][num], ascending, then KEY_NONE
    float *out;
    int *parents, *tokens;
};

struct alignas(16) BeamShared {  // the lists lie behind it
    uint32_t table[32];
    uint2 powers[32];  // c_powers: the first's bits less j 2^18, the second's
    unsigned long long red[2][BM_WARPS];
    uint32_t red_u[2 * BM_WARPS];
    unsigned long long first, dropped;  // dropped: what left the list, in units like `rest`
    int count, shrunk;
};

// A beam that is extended: its score is finite and it has not finished.
DEV bool beam_live(const BeamParams &p, int64_t row) {
    const float s = p.scores[row];
    return fabsf(s) < INFINITY && !(p.finished && p.finished[row]);
}

// A logit as it is ordered: NaN counts as -inf, -0 as +0 (they are equal: the index decides).
DEV float beam_logit(float x) { return fmaxf(x, -INFINITY) + 0.f; }

DEV float ordered_value(uint32_t o) { return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o); }
DEV float key_value(unsigned long long key) { return ordered_value(~(uint32_t)(key >> 32)); }

// 2^(j/32): the nearest fp32, and how far the power is from it, relative to it.
static __constant__ float2 c_powers[32] = {
    {1.f, 0.f}, {0x1.059b0ep+0f, -4.7084576e-08f}, {0x1.0b5586p+0f, 4.628547e-08f}, {0x1.11301ep+0f, -5.5604225e-08f},
    {0x1.172b84p+0f, -1.19921575e-08f}, {0x1.1d4874p+0f, -4.8776062e-08f}, {0x1.2387a6p+0f, 4.7297824e-08f}, {0x1.29e9ep+0f, -3.4814427e-08f},
    {0x1.306fep+0f, 3.193418e-08f}, {0x1.371a74p+0f, -2.6886665e-08f}, {0x1.3dea64p+0f, 3.6210572e-08f}, {0x1.44e086p+0f, 1.118421e-09f},
    {0x1.4bfdaep+0f, -3.099072e-08f}, {0x1.5342b6p+0f, -2.638301e-08f}, {0x1.5ab07ep+0f, -7.475213e-09f}, {0x1.6247ecp+0f, -4.2456357e-08f},
    {0x1.6a09e6p+0f, 1.7114271e-08f}, {0x1.71f75ep+0f, 2.3001967e-08f}, {0x1.7a1148p+0f, -3.0476834e-08f}, {0x1.82589ap+0f, -1.6538538e-08f},
    {0x1.8ace54p+0f, 5.233334e-09f}, {0x1.93737cp+0f, -3.5920646e-08f}, {0x1.9c4918p+0f, 6.1075918e-09f}, {0x1.a5503cp+0f, -3.1140544e-08f},
    {0x1.ae89fap+0f, -1.4719605e-08f}, {0x1.b7f77p+0f, -2.8218102e-08f}, {0x1.c199bep+0f, -5.258795e-09f}, {0x1.cb720ep+0f, -6.3603873e-09f},
    {0x1.d5818ep+0f, -6.1282597e-09f}, {0x1.dfc974p+0f, -2.4880409e-08f}, {0x1.ea4afap+0f, 5.1406093e-09f}, {0x1.f50766p+0f, -8.697267e-09f}};

// Two fp32 numbers of a register pair, an instruction for both.
struct Pair {
    unsigned long long b;
    DEV Pair() {}
    DEV Pair(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(x), "f"(y)); }
    DEV float2 both() const {
        float2 f;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(b));
        return f;
    }
};
DEV Pair pair_fma(Pair x, Pair y, Pair z) {
    Pair r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.b) : "l"(x.b), "l"(y.b), "l"(z.b));
    return r;
}
DEV Pair pair_add(Pair x, Pair y) {
    Pair r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.b) : "l"(x.b), "l"(y.b));
    return r;
}
DEV Pair operator-(Pair x, Pair y) { return pair_fma(y, Pair(-1.f, -1.f), x); }  // (exact as a subtraction is)

// Sum over the block (every thread gets it).
DEV uint32_t block_sum(uint32_t v, uint32_t *red) {
    v = __reduce_add_sync(FULL, v);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    uint32_t sum = 0;
#pragma unroll
    for (int i = 0; i < BM_WARPS; ++i) sum += red[i];
    return sum;
}

// A bound that at least `num` and at most `limit` values (ordered) reach, given
// that more than `limit` do in all; false: more than `limit` reach the bound, fewer
// than `num` exceed it.  hi and least: of the thread's values; count: of the
// block's that reach a bound.  The middle is first that of the values between the
// least and the largest, where logits lie evenly enough to be done in some five
// steps; then that of the 32-bit integers.
template <int WARPS, typename Count>
DEV bool bisect_by(uint32_t hi, uint32_t least, uint32_t &lo, int num, int limit, uint32_t *red, const Count &count) {
    const int lane = threadIdx.x % 32;
    hi = __reduce_max_sync(FULL, hi);
    least = __reduce_min_sync(FULL, least);
    __syncthreads();
    if (lane == 0) {
        red[threadIdx.x / 32] = hi;
        red[WARPS + threadIdx.x / 32] = least;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        hi = max(hi, red[i]);
        least = min(least, red[WARPS + i]);
    }
    lo = least;  // as many reach it
    for (int step = 0; lo < hi; ++step) {
        uint32_t mid = lo + (hi - lo + 1) / 2;
        if (step < 10) mid = min(max(ordered_bits(0.5f * ordered_value(lo) + 0.5f * ordered_value(hi)), lo + 1), hi);
        const int n = count(mid);
        if (n > limit) {
            lo = mid;
        } else if (n >= num) {
            lo = mid;
            return true;
        } else {
            hi = mid - 1;
        }
    }
    return false;
}
// A value of each thread, of those that reach lo.
template <int WARPS>
DEV bool bisect(uint32_t mine, uint32_t &lo, int num, int limit, uint32_t *red) {
    return bisect_by<WARPS>(mine, mine >= lo ? mine : ~0u, lo, num, limit, red, [&](uint32_t mid) { return __syncthreads_count(mine >= mid); });
}

constexpr uint32_t LEAST = 0x00800000u;  // the least value above -inf, ordered

template <bool BF16>
__global__ void __launch_bounds__(BM_THREADS, 3) beam_part_kernel(const BeamParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int E = BM_PER, VEC = BF16 ? 8 : 4, SIZE = BF16 ? 2 : 4;
    BeamShared &s = *reinterpret_cast<BeamShared *>(mk_smem);
    // behind s: the listed keys [cap], their ranks [cap]
    unsigned long long *cand = reinterpret_cast<unsigned long long *>(mk_smem + sizeof(BeamShared));
    int *ranks = reinterpret_cast<int *>(cand + p.cap);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int part = (int)(blockIdx.x % p.parts);
    const int64_t row = blockIdx.x / p.parts;
    if (!beam_live(p, row)) return;

    // the CTA's logits [first, last), VEC of a thread together, from the 16-byte boundary at or before the first
    const int first = part * p.chunk, last = min(first + p.chunk, p.vocab);
    const char *base = static_cast<const char *>(p.logits) + row * p.row_stride * SIZE;
    const int begin = first - (int)(((uintptr_t)base + (size_t)first * SIZE) % 16 / SIZE);
    const int pieces = (last - begin + BM_PIECE - 1) / BM_PIECE;
    uint4 raw[E / VEC];
    const auto load = [&](int piece) {
        const int from = begin + piece * BM_PIECE;
        if (from >= first && from + BM_PIECE <= last) {
            const uint4 *z = reinterpret_cast<const uint4 *>(base + (size_t)from * SIZE) + tid;
#pragma unroll
            for (int i = 0; i < E / VEC; ++i) raw[i] = __ldcs(z + i * BM_THREADS);
            return;
        }
#pragma unroll
        for (int i = 0; i < E / VEC; ++i) {
            const int x = from + (i * BM_THREADS + tid) * VEC;
            if (x >= first && x + VEC <= last) {
                raw[i] = __ldcs(reinterpret_cast<const uint4 *>(base + (size_t)x * SIZE));
            } else {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if constexpr (BF16) {
                        const uint16_t *z = reinterpret_cast<const uint16_t *>(base);
                        const int a = x + 2 * j;
                        const uint32_t lo = a >= first && a < last ? z[a] : 0xff80u, hi = a + 1 >= first && a + 1 < last ? z[a + 1] : 0xff80u;
                        w[j] = lo | hi << 16;
                    } else {
                        w[j] = x + j >= first && x + j < last ? reinterpret_cast<const uint32_t *>(base)[x + j] : 0xff800000u;
                    }
                }
                raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
    };
    load(0);
    if (tid < 32) {
        s.table[tid] = c_table[tid];
        s.powers[tid] = make_uint2(__float_as_uint(c_powers[tid].x) - ((uint32_t)tid << 18), __float_as_uint(c_powers[tid].y));
    }
    if (tid == 0) s.count = 0, s.dropped = 0;
    constexpr float CH = 1.44269502162933349609375f, CL = 1.92596303350011e-08f;  // log2(e)
    // All of these are the same in every thread but `rest`.
    float bound = ordered_value(LEAST);
    bool strict = false;             // num logits of lower indices that reach the bound are listed: only what exceeds it is wanted
    bool slow = false;               // logits too large for the products below
    int ref = 0, room = p.cap;       // room: entries that the list has at least
    unsigned long long rest = 0;
    // 2^(x log2(e) - ref), as a power w of 2^(1/32) and how far it is from that,
    // relative to w: x log2(e) 32 = k + g with an integer k, g in [-0.5, 0.5] from
    // log2(e) in two parts, 2^(g/32) - 1 by its series (ln 2 / 32 and so on; the
    // fourth term's mean is in the second's factor).  e^-42 below the bound is
    // nothing (-inf and NaN too).
    constexpr float ROUND = 12582912.f;  // 1.5 2^23: a sum with it is rounded to an integer; its bits shifted left by 18 are 0
    float least = 0.f, round = ROUND;    // bound - 42, ROUND - 32 ref
    const auto power = [&](float z, float &w, float &r) {
        const float x = fmaxf(z, least), t = fmaf(x, 32.f * CH, round);
        const float g = fmaf(x, 32.f * CL, fmaf(x, 32.f * CH, round - t));
        const uint2 p = s.powers[__float_as_uint(t) & 31];
        w = __uint_as_float(p.x + (__float_as_uint(t) << 18));
        r = fmaf(g, fmaf(g, fmaf(g, 1.693851e-6f, 2.3459810e-4f), 0.02166084939f), __uint_as_float(p.y));
    };
    const auto term = [&](float z) {  // in 2^-44
        float w, r;
        power(z, w, r);
        w *= 0x1p44f;
        return (unsigned long long)(__float2ll_rn(w) + __float2ll_rn(w * r));
    };
    // The terms of v, of which the largest is `most`.  Sums of w next to 2^6 of
    // that are exact with what each addition loses, which goes to the small parts'
    // sum.  Both are joined in 32-bit units of the largest (a conversion to 64 bits
    // is FP64's, which is slow).
    const auto terms = [&](const float (&v)[E], float most) {
        const float high = fmaf(fmaxf(fminf(most, bound), least), 32.f * CH, round);
        const int n = __float_as_int(high) << 18 >> 23;  // below 2^(n + 1); -62 and more
        const float c = __int_as_float((n + 133) << 23);
        Pair big(c, c), small(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            float w0, w1, r0, r1;
            power(v[i], w0, r0);
            power(v[i + 1], w1, r1);
            const Pair w(w0, w1), r(r0, r1), sum = pair_add(big, w);
            small = pair_add(pair_fma(w, r, small), w - (sum - big));
            big = sum;
        }
        const float2 a = big.both(), b = small.both();
        const int first = __float2int_rn(((a.x - c) + (a.y - c)) * __int_as_float((144 - n) << 23));  // in 2^(n - 17): exact
        const int second = __float2int_rn((b.x + b.y) * __int_as_float((157 - n) << 23));              // in 2^(n - 30)
        const long long sum = (((long long)first << 13) + second) << 14;                               // in 2^(n - 44)
        return (unsigned long long)((sum + ((1ll << -n) >> 1)) >> -n);
    };
    const auto raise_to = [&](uint32_t o) {
        bound = ordered_value(o);
        strict = true;
        slow = slow || !(fabsf(bound) <= 1e5f);
        if (!slow) {
            const int r = (int)ceilf(bound * CH);
            const auto shift = [&](unsigned long long x) { return r - ref < 64 ? x >> max(r - ref, 0) : 0; };
            rest = shift(rest);  // (a first bound below 0: nothing is summed yet)
            if (tid == 0) s.dropped = shift(s.dropped);
            ref = r;
            least = bound - 42.f;
            round = ROUND - 32.f * (float)r;
        }
    };
    // A listed logit's key; the list holds the index alone until it is first looked through.
    const auto key_at = [&](int i) {
        const unsigned long long key = cand[i];
        if (key >> 32) return key;
        const int x = (int)key;
        if constexpr (BF16) return sample_key(beam_logit(bf16_at(reinterpret_cast<const uint16_t *>(base), x)), x);
        else return sample_key(beam_logit(reinterpret_cast<const float *>(base)[x]), x);
    };
    // ranks of the listed among each other; the threads of a column share one
    const auto rank_all = [&](int n) {
        for (int i = tid; i < n; i += BM_THREADS) ranks[i] = 0;
        __syncthreads();
        int wide = 32;
        while (wide < n && wide < BM_THREADS) wide *= 2;
        for (int i = tid % wide; i < n; i += wide) {
            const unsigned long long key = cand[i];
            int before = 0;
            for (int j = tid / wide; j < n; j += BM_THREADS / wide) before += cand[j] < key;
            if (before) atomicAdd(&ranks[i], before);
        }
        __syncthreads();
    };
    // The bound up to what the listed allow, the list down to it; `hard`: down to
    // the num first, where many are equal.  Nothing here may depend on the order of
    // the list, which is that of the atomics.
    const auto shrink = [&](bool hard) {
        const int n = s.count;
        const int most = p.num + p.num / 2 + 4;
        uint32_t hi = 0, least = ~0u;
        for (int i = tid; i < n; i += BM_THREADS) {
            const unsigned long long key = key_at(i);
            cand[i] = key;
            hi = max(hi, ~(uint32_t)(key >> 32));
            least = min(least, ~(uint32_t)(key >> 32));
        }
        if (tid == 0) s.shrunk = 0;
        hard = hard && n > p.num;
        const uint32_t floor = ordered_bits(bound);
        unsigned long long last = KEY_NONE;  // the num-th key: those behind it leave
        if (hard) {
            __syncthreads();
            unsigned long long lo = 0;
            while (lo < last) {
                const unsigned long long mid = lo + (last - lo) / 2;
                uint32_t c = 0;
                for (int i = tid; i < n; i += BM_THREADS) c += cand[i] <= mid;
                if ((int)block_sum(c, s.red_u) >= p.num) last = mid;
                else lo = mid + 1;
            }
            raise_to(~(uint32_t)(last >> 32));
        } else if (n > most) {
            uint32_t lo = floor;
            bisect_by<BM_WARPS>(hi, least, lo, p.num, most, s.red_u, [&](uint32_t mid) {
                if (n <= BM_THREADS) return __syncthreads_count(hi >= mid);
                uint32_t c = 0;
                for (int i = tid; i < n; i += BM_THREADS) c += ~(uint32_t)(cand[i] >> 32) >= mid;
                return (int)block_sum(c, s.red_u);
            });
            if (lo > floor) raise_to(lo);
        }
        unsigned long long gone = 0;  // (as integers, and to one sum: which thread has which is not known)
        for (int i0 = 0; i0 < n; i0 += BM_THREADS) {
            const bool there = i0 + tid < n;
            const unsigned long long key = there ? cand[i0 + tid] : KEY_NONE;
            __syncthreads();
            if (there) {
                const float z = key_value(key);
                if (z >= bound && key <= last) cand[atomicAdd(&s.shrunk, 1)] = key;
                else if (!slow) gone += term(z);
            }
        }
        gone = warp_sum64(gone);
        if (lane == 0 && gone) atomicAdd(&s.dropped, gone);
        __syncthreads();
        if (tid == 0) s.count = s.shrunk;
        __syncthreads();
    };
    for (int piece = 0; piece < pieces; ++piece) {
        float v[E];
#pragma unroll
        for (int i = 0; i < E / VEC; ++i) {
            const uint4 w = raw[i];
            if constexpr (BF16) {
                float f[8];
                bf16x8(w, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i * VEC + j] = f[j];
            } else {
                v[4 * i] = __uint_as_float(w.x), v[4 * i + 1] = __uint_as_float(w.y);
                v[4 * i + 2] = __uint_as_float(w.z), v[4 * i + 3] = __uint_as_float(w.w);
            }
        }
        if (piece + 1 < pieces) load(piece + 1);
        const auto at = [&](int i) { return begin + piece * BM_PIECE + (i / VEC * BM_THREADS + tid) * VEC + i % VEC; };
        uint32_t want = 0;  // bit i: logit i is listed
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < E; ++i) most = fmaxf(most, v[i]);
        int threads = strict ? __syncthreads_count(most > bound) : BM_THREADS;
        float from = bound;  // logits above it are listed
        if (threads > p.limit || !strict) {  // the first piece, or one with many large logits: the bound from its own
            const uint32_t mine = ordered_bits(beam_logit(most));
            uint32_t lo = ordered_bits(bound) + (strict ? 1 : 0);
            bool found = true;
            threads = __syncthreads_count(mine >= lo);
            if (threads > p.limit) {
                found = bisect<BM_WARPS>(mine, lo, p.num, p.num + p.num / 2 + 4, s.red_u);
                raise_to(lo);
                threads = p.limit;
                if (!found) {  // many threads have the same largest logit
                    uint32_t more = 0;
#pragma unroll
                    for (int i = 0; i < E; ++i) more += v[i] > bound;
                    const int need = p.num - (int)block_sum(more, s.red_u);
                    int x = max(first, begin + piece * BM_PIECE) - 1, z = min(last, begin + (piece + 1) * BM_PIECE) - 1;
                    if (need <= 0) z = x;
                    while (z - x > 1) {  // the least index up to which `need` logits are at the bound
                        const int mid = x + (z - x) / 2;
                        uint32_t n = 0;
#pragma unroll
                        for (int i = 0; i < E; ++i) n += v[i] == bound && at(i) <= mid;
                        if ((int)block_sum(n, s.red_u) >= need) z = mid;
                        else x = mid;
                    }
#pragma unroll
                    for (int i = 0; i < E; ++i) {
                        const bool in = v[i] == bound && at(i) <= z;
                        want |= (uint32_t)in << i;
                        v[i] = in ? -INFINITY : v[i];
                    }
                }
            }
            // those at the bound too: above the next value below it (of both zeros)
            from = found ? ordered_value(lo - (lo == 0x80000000u ? 2 : 1)) : bound;
        }
        if (most > from) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const bool in = v[i] > from;
                want |= (uint32_t)in << i;
                v[i] = in ? -INFINITY : v[i];  // no term
            }
        }
        if (want) {
            int to = atomicAdd(&s.count, __popc(want));
            for (; want; want &= want - 1) cand[to++] = (uint32_t)at(__ffs(want) - 1);
        }
        if (strict && !slow) rest += terms(v, most);  // (no bound yet: all that are finite are listed)
        room -= threads * E;
        if (room < p.limit * E) {
            __syncthreads();
            shrink(false);
            room = p.cap - s.count;
            if (room < p.limit * E) {
                __syncthreads();  // the count is read
                shrink(true);
                room = p.cap - s.count;
            }
        }
    }
    __syncthreads();
    shrink(false);
    if (s.count > 512) {  // many are equal: ranking them by comparing each with all would take longer
        __syncthreads();
        shrink(true);
    }
    const int n = s.count, kept = min(n, p.num);
    rank_all(n);
    for (int i = tid; i < n; i += BM_THREADS)
        if (ranks[i] == 0) s.first = cand[i];
    __syncthreads();
    const float top = n ? key_value(s.first) : -INFINITY;
    const Weigher weigh{top, CH, CL, s.table};
    unsigned long long list = 0;
    if (!slow) {
        for (int i = tid; i < n; i += BM_THREADS) list += weigh(key_value(cand[i]));
    } else {  // products with log2(e) would lose the fraction: all by the difference from the largest
        rest = 0;
#pragma unroll 1
        for (int x = first + tid; x < last; x += BM_THREADS) {
            float z;
            if constexpr (BF16) z = bf16_at(reinterpret_cast<const uint16_t *>(base), x);
            else z = reinterpret_cast<const float *>(base)[x];
            z = beam_logit(z);
            list += z == -INFINITY ? 0 : weigh(z);
        }
    }
    list = warp_sum64(list);
    rest = warp_sum64(rest);
    if (lane == 0) {
        s.red[0][warp] = list;
        s.red[1][warp] = rest;
    }
    __syncthreads();
    unsigned long long *to = p.keys + (int64_t)blockIdx.x * p.num;
    for (int i = tid; i < n; i += BM_THREADS)
        if (ranks[i] < p.num) to[ranks[i]] = cand[i];
    for (int i = kept + tid; i < p.num; i += BM_THREADS) to[i] = KEY_NONE;
    if (tid == 0) {
        BeamPart r{top, ref, 0, slow ? 0 : s.dropped};
        for (int i = 0; i < BM_WARPS; ++i) {
            r.list += s.red[0][i];
            r.rest += s.red[1][i];
        }
        p.rows[blockIdx.x] = r;
    }
}

// fp64 totals as integers that rise with them.
DEV unsigned long long ordered64(double x) {
    const long long b = __double_as_longlong(x + 0.0);
    return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}

DEV double unordered64(unsigned long long t) {
    return __longlong_as_double(t >> 63 ? t & 0x7fffffffffffffffull : ~t);
}

// x 2^(up - d), d >= 0 in 32.32 fixed point: to 2^-34 of itself, whatever d is.
DEV unsigned long long octaves_below(unsigned long long x, long long d, int up, const uint32_t *table) {
    const unsigned long long w = octave_weight(d & 0xffffffffll, table), hi = __umul64hi(x, w), lo = x * w;
    const long long n = 44 - up + (d >> 32);  // 42 and more
    return n < 64 ? hi << (64 - n) | lo >> n : n < 128 ? hi >> (n - 64) : 0;
}

// ln(sum 2^-44) for a sum of 1 and more of them: fp32's logarithm of the
// fraction, corrected by how far its exponential is from it, so that no FP64
// function is called (one warp's takes microseconds on this GPU).
DEV double log_sum(unsigned long long sum, const uint32_t *table) {
    const int lead = 63 - __clzll(sum);
    const unsigned long long m = lead > 44 ? sum >> (lead - 44) : sum << (44 - lead);  // [1, 2) in 2^-44
    const float y = logf((float)m * 0x1p-44f);
    const Weigher weigh{0.f, 1.44269502162933349609375f, 1.92596303350011e-08f, table};
    const unsigned long long w = y > 0.f ? weigh(-y) : 1ull << 44;  // exp(-y)
    const unsigned long long prod = __umul64hi(m << 10, w << 10);   // 2^44 m exp(-y): 2^(54 + 54 - 64)
    const float r = (float)((long long)prod - (1ll << 44)) * 0x1p-44f;
    return ((double)(lead - 44) * 0.6931471805599453 + (double)y) + (double)r;
}

// By the second launch's block: the list's n candidates down to those whose value
// is at least the K-th largest, which it returns (n > K; one left of equal ones is
// all of them).  64 steps of a barrier each; the values are formed again in each of
// them (kept in registers, the rare case took half the time and the others 0.5 us more).
template <typename Value>
DEV unsigned long long narrow(int *list, int &n, int K, uint32_t *red, int &count, const Value &value) {
    const int tid = threadIdx.x;
    __syncthreads();  // `red` is read
    if (tid < 3) red[tid] = 0;
    __syncthreads();
    unsigned long long lo = 0, hi = ~0ull;  // at least K reach lo
    for (int step = 0; lo < hi; ++step) {
        const unsigned long long mid = lo + (hi - lo) / 2 + 1;
        uint32_t c = 0;
#pragma unroll 1
        for (int y = tid; y < n; y += BM_MERGE_THREADS) c += value(list[y]) >= mid;
        c = __reduce_add_sync(FULL, c);
        if (tid % 32 == 0 && c) atomicAdd(&red[step % 3], c);
        __syncthreads();
        if ((int)red[step % 3] >= K) lo = mid;
        else hi = mid - 1;
        if (tid == 0) red[(step + 2) % 3] = 0;  // the one that all have read
    }
    if (tid == 0) count = 0;
    for (int y = 0; y < n; y += BM_MERGE_THREADS) {
        const int i = y + tid < n ? list[y + tid] : -1;
        __syncthreads();
        if (i >= 0 && value(i) >= lo) list[atomicAdd(&count, 1)] = i;
    }
    __syncthreads();
    n = count;
    return lo;
}

// Candidates that a bound may let through.
__host__ __device__ constexpr int beam_limit(int num) { return num + num / 2 + 4; }

// One CTA per prompt: of all parts' candidates those with the largest totals.
__global__ void __launch_bounds__(BM_MERGE_THREADS) beam_merge_kernel(const BeamParams p) {
    const int tid = threadIdx.x, lane = tid % 32, W = p.beams, K = p.num, S = p.parts, per = S * K, all = W * per;
    double *s_add = reinterpret_cast<double *>(mk_smem);            // [64]: a beam's score less its log sum of exp(z - top)
    float *s_top = reinterpret_cast<float *>(s_add + BM_MAXBEAMS);  // [64]
    int *s_state = reinterpret_cast<int *>(s_top + BM_MAXBEAMS);    // [64]: 2 extended, 1 finished, 0 neither
    float *s_fast = reinterpret_cast<float *>(s_state + BM_MAXBEAMS);         // [64]: s_add in fp32
    uint32_t *s_table = reinterpret_cast<uint32_t *>(s_fast + BM_MAXBEAMS);   // [32]
    uint32_t *s_red = s_table + 32;                                 // [32]
    const int limit = beam_limit(K);
    unsigned long long *first = reinterpret_cast<unsigned long long *>(s_red + 32);  // [2 limit]: keys of the listed
    unsigned long long *total = first + 2 * limit;                  // [all]: ordered
    int *list = reinterpret_cast<int *>(total + all);               // [all]: those that reach the bound
    int &s_count = list[all];
    const int64_t row0 = (int64_t)blockIdx.x * W;
    if (tid == 0) s_count = 0;
    if (tid < 32) s_table[tid] = c_table[tid];
    if (tid < W) s_state[tid] = beam_live(p, row0 + tid) ? 2 : fabsf(p.scores[row0 + tid]) < INFINITY ? 1 : 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();
    const unsigned long long none = ordered64(-INFINITY);
    const auto key_of = [&](int i) {
        const int w = i / per;
        return s_state[w] == 2 ? p.keys[(row0 + w) * per + (i - w * per)]
             : s_state[w] == 1 && i == w * per ? (unsigned long long)(unsigned)p.end : KEY_NONE;  // finished: goes on as it is
    };
    const unsigned long long ahead = tid < all ? key_of(tid) : KEY_NONE;  // while the sums are formed
    // a warp per beam: its largest logit and the sum (integers: in any order)
    for (int w = tid / 32; w < W; w += BM_MERGE_THREADS / 32) {
        const float score = p.scores[row0 + w];
        if (s_state[w] != 2) {
            if (lane == 0) s_add[w] = s_fast[w] = score;
            continue;
        }
        const BeamPart *r = p.rows + (row0 + w) * S;
        float top = -INFINITY;
        for (int i = lane; i < S; i += 32) top = fmaxf(top, r[i].top);
        top = warp_max(top);
        const Weigher weigh{top, 1.44269502162933349609375f, 1.92596303350011e-08f, s_table};
        const float oh = fminf(top * weigh.ch, 0x1p20f), ol = oh < 0x1p20f ? fmaf(top, weigh.ch, -oh) + top * weigh.cl : 0.f;
        const long long octaves = __float2ll_rn(oh * 0x1p32f) + __float2ll_rn(ol * 0x1p32f);  // top log2(e)
        unsigned long long sum = 0;
        for (int i = lane; i < S && top > -INFINITY; i += 32) {
            const BeamPart x = r[i];
            if (x.top > -INFINITY) sum += octaves_below(x.list, x.top == top ? 0 : weigh.distance(x.top, 126.f), 0, s_table);
            // 2^(ref - top log2(e)): the exponent is below 2
            if (x.rest) sum += octaves_below(x.rest, max(0ll, octaves - ((long long)x.ref - 2) * (1ll << 32)), 2, s_table);
        }
        sum = warp_sum64(sum);
        if (lane == 0) {
            s_add[w] = sum ? (double)score - log_sum(sum, s_table) : 0.0;
            s_fast[w] = (float)s_add[w];
            s_top[w] = top;
        }
    }
    __syncthreads();
    // First in fp32: a total a with its error e, of which total[i] holds a - e and
    // a + e, ordered (0: not a candidate).  FP64 is slow on this GPU, so it forms the
    // few totals alone that may be among the first.
    const auto exact = [&](int w, float z) {
        const float top = s_top[w];
        return (s_state[w] == 1 || z == top ? 0.0 : (double)z - (double)top) + s_add[w];
    };
    uint32_t most = 0;  // the thread's largest a - e
    constexpr int U = 4;
    for (int i0 = tid; i0 < all; i0 += U * BM_MERGE_THREADS) {
        unsigned long long key[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * BM_MERGE_THREADS;
            key[u] = i == tid ? ahead : i < all ? key_of(i) : KEY_NONE;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = i0 + u * BM_MERGE_THREADS, w = i / per;
            if (i >= all) continue;
            uint32_t low = 0, high = 0;
            if (key[u] != KEY_NONE) {
                const float z = key_value(key[u]), top = s_top[w], c = s_fast[w];
                const float d = s_state[w] == 1 || z == top ? 0.f : z - top;
                float a = d + c, e = 0x1p-22f * (fabsf(d) + fabsf(c));  // (three roundings of 2^-24, and those of a - e and a + e)
                if (!(fabsf(a) + e < INFINITY)) {
                    const double t = exact(w, z);
                    a = (float)t, e = 0.f;
                    if (!(t > -INFINITY)) key[u] = KEY_NONE;
                }
                if (key[u] != KEY_NONE) low = ordered_bits(a - e), high = ordered_bits(a + e);
            }
            most = max(most, low);
            total[i] = (unsigned long long)high << 32 | low;
        }
    }
    // a bound that num threads' largest reach: what may reach it is listed
    uint32_t lo = 1;
    if (__syncthreads_count(most > 0) > limit) bisect<BM_MERGE_THREADS / 32>(most, lo, K, limit, s_red);
    for (int i = tid; i < all; i += BM_MERGE_THREADS)
        if ((uint32_t)(total[i] >> 32) >= lo) list[atomicAdd(&s_count, 1)] = i;
    __syncthreads();
    int n = s_count;
    // The threads' candidates have like places in their parts' lists, so that many
    // may be listed: once more among these.
    if (n > 2 * limit) {
        most = 0;
        for (int x = tid; x < n; x += BM_MERGE_THREADS) most = max(most, (uint32_t)total[list[x]]);
        if (__syncthreads_count(most >= lo) > limit) bisect<BM_MERGE_THREADS / 32>(most, lo, K, limit, s_red);
        __syncthreads();
        if (tid == 0) s_count = 0;
        for (int x0 = 0; x0 < n; x0 += BM_MERGE_THREADS) {
            const int i = x0 + tid < n ? list[x0 + tid] : -1;
            __syncthreads();
            if (i >= 0 && (uint32_t)(total[i] >> 32) >= lo) list[atomicAdd(&s_count, 1)] = i;
        }
        __syncthreads();
        n = s_count;
    }
    for (int x = tid; x < n; x += BM_MERGE_THREADS) {
        const int i = list[x];
        const unsigned long long key = key_of(i);
        total[i] = ordered64(exact(i / per, key_value(key)));
        if (x < 2 * limit) first[x] = key;
    }
    __syncthreads();
    // Of equal totals the lower beam comes first, and within a beam the key.  Where
    // that leaves many (flat rows), the list down to the K first by one after the
    // other, each by bisection.
    if (n > 2 * limit) {
        const unsigned long long least = narrow(list, n, K, s_red, s_count, [&](int i) { return total[i]; });
        const int beam = W - (int)narrow(list, n, K, s_red, s_count, [&](int i) {
                             return total[i] > least ? ~0ull : (unsigned long long)(W - i / per);
                         });
        narrow(list, n, K, s_red, s_count, [&](int i) { return total[i] > least || i / per < beam ? ~0ull : ~key_of(i); });
        for (int x = tid; x < n; x += BM_MERGE_THREADS) first[x] = key_of(list[x]);
        __syncthreads();
    }
    for (int x = tid; x < n; x += BM_MERGE_THREADS) {
        const int i = list[x], w = i / per;
        const unsigned long long t = total[i], k = first[x];
        int rank = 0;
        for (int y = 0; y < n; ++y) {
            const int j = list[y];
            const unsigned long long u = total[j];
            rank += u > t;
            if (u == t && i != j) rank += j / per < w || (j / per == w && first[y] < k);
        }
        if (rank >= K) continue;
        const int64_t to = (int64_t)blockIdx.x * K + rank;
        p.out[to] = (float)unordered64(t);
        p.parents[to] = w;
        p.tokens[to] = (int)(uint32_t)k;
    }
    for (int i = n + tid; i < K; i += BM_MERGE_THREADS) {
        const int64_t to = (int64_t)blockIdx.x * K + i;
        p.out[to] = -INFINITY;
        p.parents[to] = p.tokens[to] = -1;
    }
}

// A piece lists all logits of as many threads as may reach its bound; the list takes two such pieces and more.
static int beam_listers(int num) { return std::min(BM_THREADS, std::max(64, 2 * num)); }
static int beam_cap(int num) { return beam_listers(num) * BM_PER * 3; }
static int beam_smem(int num) { return (int)sizeof(BeamShared) + beam_cap(num) * 12; }
// CTAs that an SM holds: 3 by their registers, fewer by the lists of many continuations (a CTA takes 1024 bytes more).
static int beam_resident(int num) { return std::min(3, (SERVE_SMEM + 1024) / (beam_smem(num) + 1024)); }

// Parts of a row.  As many CTAs as the GPU holds at once (128 rows of 151,936 fp32
// logits, a cheaper sum: 29.1 us, with twice as many 36.3), no shorter parts than
// a piece, and no more candidates than the second launch holds.
static void beam_parts(const mk_beam_desc *d, int ctas, int &parts, int &chunk) {
    const int64_t rows = std::max<int64_t>(1, (int64_t)d->batch * d->beams);
    int64_t n = std::max<int64_t>(1, ctas / rows);
    n = std::min<int64_t>(n, (d->vocab + BM_PIECE - 1) / BM_PIECE);
    n = std::min<int64_t>(n, BM_CANDIDATES / (d->beams * d->num));
    chunk = (int)(((d->vocab + n - 1) / n + 7) / 8 * 8);
    parts = (d->vocab + chunk - 1) / chunk;
}

static int beam_sizes(const mk_beam_desc *d, int ctas, int &parts, int &chunk) {
    if (!d) return set_error(MK_ERR_INVALID, "null descriptor");
    if (d->batch < 0 || d->beams <= 0 || d->num <= 0 || d->vocab <= 0)
        return set_error(MK_ERR_INVALID, "batch negative, or beams, num or vocab not positive");
    if (d->beams > BM_MAXBEAMS || d->num > BM_MAXNUM) return set_error(MK_ERR_UNSUPPORTED, "more than 64 beams or 128 continuations");
    if (d->vocab > BM_MAXVOCAB) return set_error(MK_ERR_UNSUPPORTED, "vocab above 622592");
    beam_parts(d, ctas, parts, chunk);
    if ((int64_t)d->batch * d->beams * parts > INT32_MAX) return set_error(MK_ERR_UNSUPPORTED, "too many rows");
    return MK_OK;
}
static uint64_t beam_part_bytes(const mk_beam_desc *d, int parts) { return (uint64_t)d->batch * d->beams * parts * sizeof(BeamPart); }

}  // namespace mk

using namespace mk;

extern "C" {

int mk_beam_select_workspace(const mk_beam_desc *d, uint64_t *bytes) {
    if (!bytes) return set_error(MK_ERR_INVALID, "bytes is null");
    int parts, chunk;  // (on any device: fewer SMs make fewer parts)
    if (int rc = beam_sizes(d, 3 * BM_MAXSMS, parts, chunk)) return rc;
    *bytes = beam_part_bytes(d, parts) + (uint64_t)d->batch * d->beams * parts * d->num * 8;
    return MK_OK;
}

int mk_beam_select(const mk_beam_desc *d, void *workspace, uint64_t workspace_bytes, void *stream) {
    uint64_t need = 0;
    if (int rc = mk_beam_select_workspace(d, &need)) return rc;
    const int64_t rows = (int64_t)d->batch * d->beams;
    if (rows > 1 && d->row_stride < d->vocab) return set_error(MK_ERR_INVALID, "rows overlap");
    if (d->finished && (d->end < 0 || d->end >= d->vocab)) return set_error(MK_ERR_INVALID, "end is no token");
    if (rows == 0) return MK_OK;
    if (!d->logits || !d->scores || !d->out_scores || !d->parents || !d->tokens) return set_error(MK_ERR_INVALID, "null argument");
    if (d->logits % (d->bf16 ? 2 : 4) || (d->scores | d->out_scores | d->parents | d->tokens) % 4)
        return set_error(MK_ERR_INVALID, "a pointer is not aligned to its type");
    if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < need)
        return set_error(MK_ERR_INVALID, "workspace missing, unaligned (16 bytes) or too small");
    BeamParams p{};
    p.logits = reinterpret_cast<const void *>(d->logits);
    p.row_stride = d->row_stride;
    p.vocab = d->vocab;
    p.beams = d->beams;
    p.num = d->num;
    p.scores = reinterpret_cast<const float *>(d->scores);
    p.finished = reinterpret_cast<const uint8_t *>(d->finished);
    p.end = d->end;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return serve_cuda_fail(e, "device query");
    beam_parts(d, std::min(sms, BM_MAXSMS) * beam_resident(d->num), p.parts, p.chunk);
    p.rows = static_cast<BeamPart *>(workspace);
    p.keys = reinterpret_cast<unsigned long long *>(static_cast<uint8_t *>(workspace) + beam_part_bytes(d, p.parts));
    p.out = reinterpret_cast<float *>(d->out_scores);
    p.parents = reinterpret_cast<int *>(d->parents);
    p.tokens = reinterpret_cast<int *>(d->tokens);
    p.limit = beam_listers(d->num);
    p.cap = beam_cap(d->num);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    void (*f)(const BeamParams) = d->bf16 ? beam_part_kernel<true> : beam_part_kernel<false>;
    static std::atomic<uint32_t> ready[SERVE_MAX_DEVICES];
    if (int rc = serve_prepare(reinterpret_cast<const void *>(f), ready, d->bf16 ? 1 : 0, false)) return rc;
    if (int rc = serve_prepare(reinterpret_cast<const void *>(beam_merge_kernel), ready, 2, false)) return rc;
    f<<<(unsigned)(rows * p.parts), BM_THREADS, beam_smem(d->num), st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return serve_cuda_fail(e, "beam selection launch");
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)d->batch);
    cfg.blockDim = dim3(BM_MERGE_THREADS);
    cfg.dynamicSmemBytes = BM_MAXBEAMS * 20 + 64 * 4 + 2 * beam_limit(p.num) * 8 + p.beams * p.parts * p.num * 12 + 4;
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, beam_merge_kernel, (const BeamParams)p);
    return e == cudaSuccess ? MK_OK : serve_cuda_fail(e, "beam merge launch");
}

}  // extern "C"
