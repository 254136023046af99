// Attention of new tokens over an 8-bit paged KV cache.
//
// Mathematics.  One pass over a sequence's pages with the running maximum m
// and sum l of the softmax (in log2 units); partial results of page ranges
// merge as sum_i 2^(m_i - M) (l_i, O_i).  All sums are fp32.
//
// What bounds it: the cache's bytes, 2 D per token and kv head, each read
// once; a group of q heads (and of new tokens) shares them.
//
// Matrix products.  Codes go to the tensor cores as they lie in memory
// (mma.sync m16n8k32, e4m3 x e4m3 -> fp32): converting them to f16 first
// would cost as many conversions as the SM can issue at the HBM rate.  A
// bf16 query is exactly the sum of two e4m3 numbers at scales 1 and 1/16 (8
// significant bits = 4 + 4; its row is scaled by a power of two into e4m3's
// range), and a probability is one to 2^-8 of its value; the two halves are
// rows g and g + 8 of the 16-row tile, so that both products of a row land
// in the same thread: c[0..1] + c[2..3] / 16.  The 8 rows of a tile are q
// heads of one kv head, then new tokens.  Against tcgen05: its least tile is
// 64 rows, a decode step fills 4 to 8 of them, and the kernel is bound by
// bytes either way.
//
// Token order.  A contraction may run over tokens in any order, so column n
// of score tile j is token (P/4)(n/2) + 2j + n%2 of the page: then thread t
// of a quad owns the P/4 tokens from (P/4) t on, its probabilities already
// are the second product's A fragment, and its V operand is one P/4-byte run
// of a transposed V row.
//
// Work split.  The pages of all (sequence, row tile, kv head) form one axis,
// cut into equal ranges, one per CTA (one CTA per SM): ragged batches and
// single long sequences balance alike.  A producer warp streams the pages
// through a shared-memory ring with bulk copies; warps of a tile take every
// (8 / tiles)-th page and merge in shared memory.  A unit that one CTA covers
// is written at once; ranges cut by a CTA boundary go to the workspace and a
// second small launch (dependent launch, so that its start overlaps) merges
// them in order: results do not depend on timing.
#include <algorithm>
#include <climits>

#include "dev_serve.cuh"

namespace mk {

constexpr int ATT_WARPS = 8;                        // consumer warps
constexpr int ATT_THREADS = (ATT_WARPS + 1) * 32;   // + the producer
constexpr int ATT_MAXB = 1024;                      // sequences per call
constexpr int ATT_MAXSTAGES = 32;

struct AttParams {
    CacheView c;  // of the layer: k, v, ks, vs point at it
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    int64_t qs_t, qs_h, os_t, os_h;
    const int *table, *lens, *q_start;
    int batch, width, group, tokens, max_tokens, window, stages, ctas;
    float scale_log2;
    // workspace: prefix int64 [batch + 1]; partial (m, l) [ctas][2][RT][2]; partial O [ctas][2][RT][D]
    long long *prefix;
    float *part_ml, *part_o;
};

// What a sequence asks for: its query rows, its pages [lo, hi) that any row sees.
struct AttSeq {
    int q0, cnt, len, lo, hi;
};

template <int P>
DEV AttSeq att_seq(const AttParams &p, int b, bool report) {
    AttSeq s;
    s.len = p.lens[b];
    s.q0 = p.q_start ? p.q_start[b] : b * p.max_tokens;
    s.cnt = (p.q_start ? p.q_start[b + 1] : s.q0 + p.max_tokens) - s.q0;
    if (s.q0 < 0 || s.cnt < 0 || s.q0 > p.tokens || s.cnt > p.tokens - s.q0) {  // its rows are not known: none
        if (report) note_failure(p.c.status, MK_ERR_DEVICE_CHECK, b, s.q0, -1);
        s.q0 = s.cnt = s.len = s.lo = s.hi = 0;
        return s;
    }
    if (s.len < 0 || (int64_t)s.len > (int64_t)p.width * P) {
        if (report) note_failure(p.c.status, MK_ERR_DEVICE_CHECK, b, s.len, -1);
        s.len = 0;
    }
    s.hi = (s.len + P - 1) / P;
    const int64_t first = (int64_t)s.len - s.cnt - p.window + 1;
    s.lo = p.window > 0 && first > 0 ? min((int)(first / P), s.hi) : 0;
    return s;
}

// CTAs that get work: every one of them at least a page.
DEV int att_used(long long total, int ctas) { return (int)min((long long)ctas, total); }
// CTA of work item x when `total` items are cut into `ctas` <= total ranges [c total / ctas, (c + 1) total / ctas).
DEV int att_owner(long long x, long long total, int ctas) { return (int)(((x + 1) * ctas - 1) / total); }

// One range of pages of one unit, as every warp of the CTA walks them.
struct AttSeg {
    int b, tile, h, p0, p1;   // pages [p0, p1)
    int q0, cnt, len;
    bool whole;               // the unit's every page
    bool first;               // the CTA's first range
};

struct AttShared {
    long long *prefix;  // [batch + 1]
    float2 *scale;      // [stages]: (K scale, V scale), K scale < 0: page not loaded
    uint64_t *full, *empty;
    float *merge;       // [8 warps][8 rows][D + 8]
    float *ml;          // [8 warps][8 rows][2]
    int *ctrl;          // [0] abort
    uint8_t *ring;
};

template <int D>
__host__ __device__ constexpr int att_fixed_bytes() {
    return ATT_WARPS * 8 * (D + 8) * 4 + ATT_WARPS * 8 * 2 * 4 + ATT_MAXSTAGES * (8 + 16) + 16;
}

template <int D>
DEV AttShared att_shared(const AttParams &p) {
    AttShared s;
    uint8_t *at = mk_smem;
    s.full = reinterpret_cast<uint64_t *>(at);
    s.empty = s.full + ATT_MAXSTAGES;
    at += ATT_MAXSTAGES * 16;
    s.scale = reinterpret_cast<float2 *>(at);
    at += ATT_MAXSTAGES * 8;
    s.ctrl = reinterpret_cast<int *>(at);
    at += 16;
    s.ml = reinterpret_cast<float *>(at);
    at += ATT_WARPS * 8 * 2 * 4;
    s.merge = reinterpret_cast<float *>(at);
    at += ATT_WARPS * 8 * (D + 8) * 4;
    s.prefix = reinterpret_cast<long long *>(at);
    const uint32_t used = (uint32_t)(at - mk_smem) + (p.batch + 1) * 8;
    s.ring = mk_smem + ((used + 127) & ~127u);
    return s;
}

// Walks the ranges of this CTA; the same in every warp.
template <int P, int RT>
struct AttWalk {
    const AttParams &p;
    const long long *prefix;
    long long x, end;
    int b;
    bool first = true;
    DEV AttWalk(const AttParams &p_, const long long *pre) : p(p_), prefix(pre) {
        const long long total = pre[p.batch];
        const int ctas = max(1, att_used(total, p.ctas));
        x = end = 0;
        if ((int)blockIdx.x < ctas) {
            x = (long long)blockIdx.x * total / ctas;
            end = (long long)(blockIdx.x + 1) * total / ctas;
        }
        int a = 0, z = p.batch;  // the last b with prefix[b] <= x
        while (z - a > 1) {
            const int mid = (a + z) / 2;
            if (pre[mid] <= x) a = mid;
            else z = mid;
        }
        b = a;
    }
    DEV bool next(AttSeg &g) {
        if (x >= end) return false;
        while (prefix[b + 1] <= x) ++b;
        const AttSeq s = att_seq<P>(p, b, false);
        const int np = s.hi - s.lo;
        const long long r = x - prefix[b];
        const int unit = (int)(r / np), pg = (int)(r % np);
        const int n = (int)min((long long)(np - pg), end - x);
        x += n;
        g.b = b;
        g.tile = unit / p.c.hkv;
        g.h = unit % p.c.hkv;
        g.q0 = s.q0;
        g.cnt = s.cnt;
        g.len = s.len;
        g.whole = n == np;
        g.first = first;
        first = false;
        // the tile's own rows may see fewer pages than the sequence's
        const int rows = s.cnt * p.group;
        const int i0 = g.tile * RT / p.group, i1 = (min((g.tile + 1) * RT, rows) - 1) / p.group;
        const int top = s.len - s.cnt + i1, bottom = s.len - s.cnt + i0;
        const int seen_hi = top < 0 ? 0 : top / P + 1;
        const int seen_lo = p.window > 0 ? max(0, bottom - p.window + 1) / P : 0;
        g.p0 = max(s.lo + pg, seen_lo);
        g.p1 = min(s.lo + pg + n, seen_hi);
        return true;
    }
};

// Bounded wait on a ring barrier (a few seconds): false if it ran out or
// another warp gave up.
DEV bool att_wait(const AttParams &p, const AttShared &s, uint64_t *bar, uint32_t parity) {
    if (mbar_test(bar, parity)) return true;
    for (int i = 0; i < 4000; ++i) {
        if (mbar_wait_hint(bar, parity, 1000000)) return true;
        if (*reinterpret_cast<volatile int *>(s.ctrl)) return false;
    }
    note_failure(p.c.status, MK_ERR_TIMEOUT, -1, blockIdx.x, -1);
    *reinterpret_cast<volatile int *>(s.ctrl) = 1;
    return false;
}

template <int D, int P, int MT>
DEV void att_produce(const AttParams &p, const AttShared &s) {
    constexpr int RT = 8 * MT, PAGE = P * D;
    const int lane = threadIdx.x % 32;
    AttWalk<P, RT> walk(p, s.prefix);
    AttSeg g;
    int it = 0;
    bool ok = true;
    while (ok && walk.next(g)) {
        for (int base = g.p0; ok && base < g.p1; base += 32) {
            const int n = min(32, g.p1 - base);
            int id = -1;
            float ks = -1.f, vs = 0.f;
            if (lane < n) {
                id = p.table[(size_t)g.b * p.width + base + lane];
                if ((unsigned)id < (unsigned)p.c.pages) {
                    ks = p.c.ks[(size_t)id * p.c.hkv + g.h];
                    vs = p.c.vs[(size_t)id * p.c.hkv + g.h];
                } else {
                    note_failure(p.c.status, MK_ERR_DEVICE_CHECK, g.b, (base + lane) * P, id);
                    id = -1;
                }
            }
            for (int i = 0; i < n; ++i, ++it) {
                const int page = __shfl_sync(FULL, id, i);
                const float k1 = __shfl_sync(FULL, ks, i), v1 = __shfl_sync(FULL, vs, i);
                const int st = it % p.stages;
                if (it >= p.stages) ok = att_wait(p, s, &s.empty[st], ((it / p.stages) & 1) ^ 1);
                ok = __shfl_sync(FULL, ok, 0);
                if (!ok) break;
                if (lane == 0) {
                    s.scale[st] = make_float2(page < 0 ? -1.f : k1, v1);
                    if (page < 0) {
                        mbar_arrive(&s.full[st]);
                    } else {
                        mbar_expect_tx(&s.full[st], 2 * PAGE);
                        const size_t off = ((size_t)page * p.c.hkv + g.h) * PAGE;
                        bulk_g2s_plain(s.ring + (size_t)st * 2 * PAGE, p.c.k + off, PAGE, &s.full[st]);
                        bulk_g2s_plain(s.ring + (size_t)st * 2 * PAGE + PAGE, p.c.v + off, PAGE, &s.full[st]);
                    }
                }
                __syncwarp();
            }
        }
    }
    if (!ok && lane == 0) {  // given up: let the copies in flight land before the CTA ends
        for (int k = max(0, it - p.stages); k < it; ++k)
            for (int i = 0; i < 200 && !mbar_wait_hint(&s.full[k % p.stages], (k / p.stages) & 1, 1000000); ++i) {
            }
    }
}

DEV void att_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
DEV float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Bytes of w that are e4m3's NaN codes (0x7f, 0xff), as a byte mask.
DEV uint32_t nan_bytes(uint32_t w) {
    const uint32_t m = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
    return m * 0xffu;
}

// The query fragment of one row: dims h2 * 64 + 16 t .. + 15, split into e4m3
// halves; returns 2^-k of the row's scaling (NaN if the row is not finite).
template <int D>
DEV float att_load_q(const uint16_t *row, int t, uint32_t (&qa)[D / 32][4]) {
    float f[D / 64][16];
    uint32_t big = 0;
#pragma unroll
    for (int h2 = 0; h2 < D / 64; ++h2) {
        uint4 x[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
        if (row) {
            x[0] = __ldg(reinterpret_cast<const uint4 *>(row + h2 * 64 + 16 * t));
            x[1] = __ldg(reinterpret_cast<const uint4 *>(row + h2 * 64 + 16 * t) + 1);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                f[h2][8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                f[h2][8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
                big = max(big, max((w[j] << 16) & 0x7fffffffu, w[j] & 0x7fff0000u));
            }
        }
    }
    big = max(big, __shfl_xor_sync(FULL, big, 1));
    big = max(big, __shfl_xor_sync(FULL, big, 2));
    // times 2^(7 - exponent) (bits 127 + 7 - (field - 127)): the row's largest value lands in [128, 256)
    const int up = min(max(261 - (int)(big >> 23), 1), 253);
    const float sc = __uint_as_float((uint32_t)up << 23);
#pragma unroll
    for (int h2 = 0; h2 < D / 64; ++h2)
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // 4 dims: a register of hi codes and one of lo codes
            uint32_t hi = 0, lo = 0;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float a = f[h2][4 * i + 2 * j] * sc, b = f[h2][4 * i + 2 * j + 1] * sc;
                const uint32_t e = to_e4m3x2(a, b);
                float ea, eb;
                half2_floats(e4m3x2_to_half2(e), ea, eb);
                hi |= e << (16 * j);
                lo |= to_e4m3x2((a - ea) * 16.f, (b - eb) * 16.f) << (16 * j);
            }
            qa[2 * h2 + i / 2][(i % 2) * 2] = hi;
            qa[2 * h2 + i / 2][(i % 2) * 2 + 1] = lo;
        }
    return big >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(254 - up) << 23);
}

DEV void att_consumer_bar() { asm volatile("bar.sync 1, %0;" ::"n"(ATT_WARPS * 32) : "memory"); }

template <int D, int P, int MT>
DEV void att_consume(const AttParams &p, const AttShared &s) {
    constexpr int RT = 8 * MT, NG = ATT_WARPS / MT, PAGE = P * D, NJ = P / 8, RUN = P / 4;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g8 = lane / 4, t = lane % 4;
    const int mt = warp % MT, grp = warp / MT;
    AttWalk<P, RT> walk(p, s.prefix);
    AttSeg g;
    int it = 0;
    bool ok = true;
    while (walk.next(g)) {
        const int rows = g.cnt * p.group;
        const int r = g.tile * RT + mt * 8 + g8;                    // this thread's row
        const int tok = r / p.group, head = g.h * p.group + r % p.group;
        const int pos = r < rows ? g.len - g.cnt + tok : -1;        // it sees [least, pos]
        const int least = p.window > 0 ? max(0, pos - p.window + 1) : 0;
        uint32_t qa[D / 32][4];
        const uint16_t *qrow = r < rows ? p.q + (int64_t)(g.q0 + tok) * p.qs_t + (int64_t)head * p.qs_h : nullptr;
        const float qf = att_load_q<D>(qrow, t, qa) * p.scale_log2;
        // pages that every row of the warp's tile sees whole need no masks
        const int all_hi = __reduce_min_sync(FULL, r < rows ? pos : INT_MAX);
        const int all_lo = __reduce_max_sync(FULL, r < rows ? least : 0);
        float m = -INFINITY, l = 0.f, o[D / 8][2];
#pragma unroll
        for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = 0.f;
        for (int pg = g.p0; pg < g.p1; ++pg, ++it) {
            if (it % NG != grp || !ok) continue;
            const int st = it % p.stages;
            ok = att_wait(p, s, &s.full[st], (it / p.stages) & 1);
            ok = __all_sync(FULL, ok);
            if (!ok) continue;
            const float2 sc = s.scale[st];
            const uint8_t *kp = s.ring + (size_t)st * 2 * PAGE, *vp = kp + PAGE;
            if (sc.x >= 0.f || sc.x != sc.x) {
                float c[NJ][4];
#pragma unroll
                for (int j = 0; j < NJ; ++j) c[j][0] = c[j][1] = c[j][2] = c[j][3] = 0.f;
#pragma unroll
                for (int h2 = 0; h2 < D / 64; ++h2)
#pragma unroll
                    for (int j = 0; j < NJ; ++j) {
                        const int row = RUN * (g8 >> 1) + 2 * j + (g8 & 1);
                        const uint4 kk = *reinterpret_cast<const uint4 *>(kp + row * D + h2 * 64 + 16 * t);
                        att_mma(c[j], qa[2 * h2], kk.x, kk.y);
                        att_mma(c[j], qa[2 * h2 + 1], kk.z, kk.w);
                    }
                const float f = sc.x * qf;
                const int first = pg * P + RUN * t;  // token of c[0][0]
                const bool edge = pg * P < all_lo || pg * P + P - 1 > all_hi;
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < NJ; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float z = fmaf(c[j][e + 2], 0.0625f, c[j][e]) * f;
                        if (edge && (first + 2 * j + e > pos || first + 2 * j + e < least)) z = -INFINITY;
                        c[j][e] = z;
                        mx = fmaxf(mx, z);
                    }
                mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 2));
                const float mn = fmaxf(m, mx), mu = mn == -INFINITY ? 0.f : mn;
                const float alpha = exp2_fast(m - mu);
                m = mn;
                // probabilities x 2^8 (e4m3's upper range), in e4m3 halves
                uint32_t pa[P / 32][4];
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < P / 32; ++k)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t hi = 0, lo = 0;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int j = 4 * k + 2 * q + i;
                            const float a = exp2_fast(c[j][0] - mu + 8.f), b = exp2_fast(c[j][1] - mu + 8.f);
                            sum += a + b;
                            uint32_t h2;
                            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h2) : "f"(b), "f"(a));
                            const uint32_t e = half2_to_e4m3x2(h2);
                            hi |= e << (16 * i);
                            // the remainder is exact in f16; x 16
                            lo |= half2_to_e4m3x2(half2_mul(half2_sub(h2, e4m3x2_to_half2(e)), 0x4c004c00u)) << (16 * i);
                        }
                        pa[k][2 * q] = hi;
                        pa[k][2 * q + 1] = lo;
                    }
                l = fmaf(l, alpha, sum);
                if (!edge) {
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        float a[4] = {0.f, 0.f, 0.f, 0.f};
                        if constexpr (P == 64) {
                            const uint4 vv = *reinterpret_cast<const uint4 *>(vp + (n * 8 + g8) * P + RUN * t);
                            att_mma(a, pa[0], vv.x, vv.y);
                            att_mma(a, pa[1], vv.z, vv.w);
                        } else {
                            const uint2 vv = *reinterpret_cast<const uint2 *>(vp + (n * 8 + g8) * P + RUN * t);
                            att_mma(a, pa[0], vv.x, vv.y);
                        }
                        o[n][0] = fmaf(fmaf(a[2], 0.0625f, a[0]), sc.y, o[n][0] * alpha);
                        o[n][1] = fmaf(fmaf(a[3], 0.0625f, a[1]), sc.y, o[n][1] * alpha);
                    }
                } else {
                    // A masked token's weight is 0, but 0 x NaN is NaN: NaN
                    // codes are taken out, and a second product of the mask
                    // with their places says which sums really contain one.
                    uint32_t see[P / 32][4];
#pragma unroll
                    for (int k = 0; k < P / 32; ++k)
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            uint32_t w = 0;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int x = first + 8 * k + 4 * q + i;
                                if (x <= pos && x >= least) w |= 0x38u << (8 * i);  // 1.0
                            }
                            see[k][2 * q] = w;
                            see[k][2 * q + 1] = 0;
                        }
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        uint32_t vv[RUN / 4], bad = 0;
#pragma unroll
                        for (int i = 0; i < RUN / 4; ++i) {
                            vv[i] = *reinterpret_cast<const uint32_t *>(vp + (n * 8 + g8) * P + RUN * t + 4 * i);
                            bad |= nan_bytes(vv[i]);
                        }
                        float a[4] = {0.f, 0.f, 0.f, 0.f}, z[4] = {0.f, 0.f, 0.f, 0.f};
                        if (__any_sync(FULL, bad != 0)) {
                            uint32_t at[RUN / 4];
#pragma unroll
                            for (int i = 0; i < RUN / 4; ++i) {
                                const uint32_t nb = nan_bytes(vv[i]);
                                vv[i] &= ~nb;
                                at[i] = nb & 0x38383838u;
                            }
#pragma unroll
                            for (int k = 0; k < P / 32; ++k) att_mma(z, see[k], at[2 * k], at[2 * k + 1]);
                        }
#pragma unroll
                        for (int k = 0; k < P / 32; ++k) att_mma(a, pa[k], vv[2 * k], vv[2 * k + 1]);
                        const float nan = __uint_as_float(0x7fc00000u);
                        o[n][0] = fmaf(fmaf(a[2], 0.0625f, a[0]), sc.y, o[n][0] * alpha) + (z[0] > 0.f ? nan : 0.f);
                        o[n][1] = fmaf(fmaf(a[3], 0.0625f, a[1]), sc.y, o[n][1] * alpha) + (z[1] > 0.f ? nan : 0.f);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.empty[st]);
        }
        l += __shfl_xor_sync(FULL, l, 1);
        l += __shfl_xor_sync(FULL, l, 2);
        // merge the NG warps of each tile
        float *mo = s.merge + (warp * 8 + g8) * (D + 8);
#pragma unroll
        for (int n = 0; n < D / 8; ++n) *reinterpret_cast<float2 *>(mo + 8 * n + 2 * t) = make_float2(o[n][0], o[n][1]);
        if (t == 0) *reinterpret_cast<float2 *>(s.ml + (warp * 8 + g8) * 2) = make_float2(m, l);
        att_consumer_bar();
        for (int i = threadIdx.x; i < RT * (D / 4); i += ATT_WARPS * 32) {
            const int row = i / (D / 4), d4 = i % (D / 4);
            float big = -INFINITY;
#pragma unroll
            for (int k = 0; k < NG; ++k) big = fmaxf(big, s.ml[((k * MT + row / 8) * 8 + row % 8) * 2]);
            const float mu = big == -INFINITY ? 0.f : big;
            float sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < NG; ++k) {
                const int w = (k * MT + row / 8) * 8 + row % 8;
                const float a = exp2_fast(s.ml[w * 2] - mu);
                const float4 x = *reinterpret_cast<const float4 *>(s.merge + w * (D + 8) + 4 * d4);
                sum = fmaf(a, s.ml[w * 2 + 1], sum);
                acc.x = fmaf(a, x.x, acc.x);
                acc.y = fmaf(a, x.y, acc.y);
                acc.z = fmaf(a, x.z, acc.z);
                acc.w = fmaf(a, x.w, acc.w);
            }
            const int rr = g.tile * RT + row;
            if (rr >= rows) continue;
            if (g.whole) {
                const int64_t token = g.q0 + rr / p.group;
                const int hd = g.h * p.group + rr % p.group;
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                *reinterpret_cast<uint2 *>(p.out + token * p.os_t + (int64_t)hd * p.os_h + 4 * d4) =
                    make_uint2(bf16_pair(acc.x * inv, acc.y * inv), bf16_pair(acc.z * inv, acc.w * inv));
                if (p.lse && d4 == 0)
                    p.lse[token * (p.group * p.c.hkv) + hd] =
                        sum == 0.f ? -INFINITY : (big - 8.f + log2f(sum)) * 0.6931471805599453f;
            } else {
                const size_t slot = ((size_t)blockIdx.x * 2 + (g.first ? 0 : 1)) * RT + row;
                *reinterpret_cast<float4 *>(p.part_o + slot * D + 4 * d4) = acc;
                if (d4 == 0) *reinterpret_cast<float2 *>(p.part_ml + slot * 2) = make_float2(big, sum);
            }
        }
        att_consumer_bar();
    }
}

template <int D, int P, int MT>
__global__ void __launch_bounds__(ATT_THREADS, 1) cache_attend_kernel(const AttParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    const AttShared s = att_shared<D>(p);
    const int tid = threadIdx.x;
    constexpr int RT = 8 * MT;
    for (int b = tid; b < p.batch; b += ATT_THREADS) {
        const AttSeq q = att_seq<P>(p, b, blockIdx.x == 0);
        s.prefix[b + 1] = (long long)((q.cnt * p.group + RT - 1) / RT) * (q.hi - q.lo) * p.c.hkv;
    }
    if (tid == 0) {
        s.prefix[0] = 0;
        s.ctrl[0] = 0;
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], MT);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (tid < 32) {  // running sums, 32 sequences at a time
        long long carry = 0;
        for (int b0 = 0; b0 < p.batch; b0 += 32) {
            const int b = b0 + tid;
            long long v = b < p.batch ? s.prefix[b + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(FULL, v, o);
                if (tid >= o) v += u;
            }
            v += carry;
            if (b < p.batch) s.prefix[b + 1] = v;
            carry = __shfl_sync(FULL, v, 31);
        }
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int b = tid; b <= p.batch; b += ATT_THREADS) p.prefix[b] = s.prefix[b];
    if (tid >= ATT_WARPS * 32) att_produce<D, P, MT>(p, s);
    else att_consume<D, P, MT>(p, s);
}

// One warp per query row: rows that see nothing get zeros, rows whose pages
// two or more CTAs shared are merged, in the order of the CTAs; the others
// are written already.
template <int D, int P>
__global__ void __launch_bounds__(256) cache_attend_merge(const AttParams p, int rt) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x % 32, heads = p.group * p.c.hkv;
    const int64_t w = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
    if (w >= (int64_t)p.tokens * heads) return;
    const int token = (int)(w / heads), head = (int)(w % heads);
    int b;
    if (p.q_start) {
        int a = 0, z = p.batch;  // the last b with q_start[b] <= token
        while (z - a > 1) {
            const int mid = (a + z) / 2;
            if (p.q_start[mid] <= token) a = mid;
            else z = mid;
        }
        b = a;
    } else {
        b = token / p.max_tokens;
        if (b >= p.batch) return;
    }
    const AttSeq s = att_seq<P>(p, b, false);
    if (token < s.q0 || token >= s.q0 + s.cnt) return;
    const int np = s.hi - s.lo, h = head / p.group, r = (token - s.q0) * p.group + head % p.group;
    constexpr int V = D / 32;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    float big = -INFINITY, sum = 0.f;
    if (np > 0) {
        const long long total = p.prefix[p.batch], x0 = p.prefix[b] + ((long long)(r / rt) * p.c.hkv + h) * np;
        const int ctas = att_used(total, p.ctas);
        const int c0 = att_owner(x0, total, ctas), c1 = att_owner(x0 + np - 1, total, ctas);
        if (c0 == c1) return;
        for (int c = c0; c <= c1; ++c) {
            // the unit is the CTA's first range unless it begins inside the CTA's
            const int k = c == c0 && x0 > (long long)c * total / ctas ? 1 : 0;
            const size_t slot = ((size_t)c * 2 + k) * rt + r % rt;
            const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + slot * 2);
            const float top = fmaxf(big, ml.x), mu = top == -INFINITY ? 0.f : top;
            const float a = exp2_fast(big - mu), e = exp2_fast(ml.x - mu);
            big = top;
            sum = fmaf(sum, a, ml.y * e);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(acc[i], a, p.part_o[slot * D + lane * V + i] * e);
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t *dst = p.out + (int64_t)token * p.os_t + (int64_t)head * p.os_h + lane * V;
#pragma unroll
    for (int i = 0; i < V; i += 2) *reinterpret_cast<uint32_t *>(dst + i) = bf16_pair(acc[i] * inv, acc[i + 1] * inv);
    if (p.lse && lane == 0)
        p.lse[w] = sum == 0.f ? -INFINITY : (big - 8.f + log2f(sum)) * 0.6931471805599453f;
}

struct AttPlan {
    int rt, ctas;
    uint64_t prefix_bytes, ml_bytes, o_bytes;
};

static int att_plan(const mk_cache_desc *c, const mk_attend_desc *a, AttPlan &pl) {
    if (!c || !a) return set_error(MK_ERR_INVALID, "null descriptor");
    if (a->batch < 0 || a->tokens < 0 || a->max_tokens < 0 || a->table_width <= 0)
        return set_error(MK_ERR_INVALID, "negative batch, tokens or max_tokens, or an empty table");
    if (a->batch > ATT_MAXB) return set_error(MK_ERR_UNSUPPORTED, "more than 1024 sequences in one call");
    if (c->kv_heads <= 0 || a->q_heads <= 0 || a->q_heads % c->kv_heads)
        return set_error(MK_ERR_INVALID, "q_heads must be a multiple of kv_heads");
    if ((int64_t)a->tokens * a->q_heads > INT32_MAX || (int64_t)a->table_width * c->page_tokens > INT32_MAX)
        return set_error(MK_ERR_UNSUPPORTED, "more than 2^31 query rows or positions");
    if (!a->q_start && (int64_t)a->batch * a->max_tokens != a->tokens)
        return set_error(MK_ERR_INVALID, "tokens must be batch x max_tokens without q_start");
    int sms = a->num_sms;
    if (sms <= 0) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return serve_cuda_fail(e, "device query");
    }
    // row tiles of 8, 16, 32 or 64 rows: the least that takes a sequence's rows of one kv head
    const int64_t rows = (int64_t)std::max(1, std::min(a->max_tokens, a->tokens)) * (a->q_heads / c->kv_heads);
    pl.rt = rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
    pl.ctas = sms;
    pl.prefix_bytes = ((uint64_t)(a->batch + 1) * 8 + 255) / 256 * 256;
    pl.ml_bytes = ((uint64_t)sms * 2 * pl.rt * 8 + 255) / 256 * 256;
    pl.o_bytes = (uint64_t)sms * 2 * pl.rt * c->head_dim * 4;
    return MK_OK;
}

using AttFn = void (*)(const AttParams);
template <int D, int P>
static AttFn att_kernel(int rt) {
    return rt == 8 ? cache_attend_kernel<D, P, 1> : rt == 16 ? cache_attend_kernel<D, P, 2>
         : rt == 32 ? cache_attend_kernel<D, P, 4> : cache_attend_kernel<D, P, 8>;
}

}  // namespace mk

using namespace mk;

extern "C" {

int mk_cache_attend_workspace(const mk_cache_desc *cache, const mk_attend_desc *attend, uint64_t *bytes) {
    AttPlan pl;
    if (!bytes) return set_error(MK_ERR_INVALID, "bytes is null");
    if (int rc = att_plan(cache, attend, pl)) return rc;
    *bytes = pl.prefix_bytes + pl.ml_bytes + pl.o_bytes;
    return MK_OK;
}

int mk_cache_attend(const mk_cache_desc *cache, int layer, const mk_attend_desc *a, void *workspace,
                    uint64_t workspace_bytes, void *stream) {
    AttParams p{};
    AttPlan pl;
    if (int rc = cache_check(cache, p.c)) return rc;
    if (int rc = att_plan(cache, a, pl)) return rc;
    if (layer < 0 || layer >= cache->layers) return set_error(MK_ERR_INVALID, "layer out of range");
    if (a->window < 0 || !(a->scale >= 0.f) || a->scale > 3e38f)
        return set_error(MK_ERR_INVALID, "window must not be negative, scale finite and not negative");
    if (a->batch == 0 || a->tokens == 0) return MK_OK;
    if (!a->q || !a->out || !a->table || !a->lens) return set_error(MK_ERR_INVALID, "null argument");
    if (a->q % 16 || a->out % 16 || a->lse % 4) return set_error(MK_ERR_INVALID, "q and out must be 16-byte aligned");
    for (int i = 0; i < 2; ++i)
        if (a->q_stride[i] % 8 || a->out_stride[i] % 8)
            return set_error(MK_ERR_INVALID, "q and out strides must be multiples of 8 elements");
    if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < pl.prefix_bytes + pl.ml_bytes + pl.o_bytes)
        return set_error(MK_ERR_INVALID, "workspace missing, unaligned (16 bytes) or too small");
    const int D = cache->head_dim, P = cache->page_tokens;
    const size_t layer_rows = (size_t)layer * cache->pages * cache->kv_heads;
    p.c.k += layer_rows * P * D;
    p.c.v += layer_rows * P * D;
    p.c.ks += layer_rows;
    p.c.vs += layer_rows;
    p.q = reinterpret_cast<const uint16_t *>(a->q);
    p.out = reinterpret_cast<uint16_t *>(a->out);
    p.lse = reinterpret_cast<float *>(a->lse);
    p.qs_t = a->q_stride[0];
    p.qs_h = a->q_stride[1];
    p.os_t = a->out_stride[0];
    p.os_h = a->out_stride[1];
    p.table = reinterpret_cast<const int *>(a->table);
    p.lens = reinterpret_cast<const int *>(a->lens);
    p.q_start = reinterpret_cast<const int *>(a->q_start);
    p.batch = a->batch;
    p.width = a->table_width;
    p.group = a->q_heads / cache->kv_heads;
    p.tokens = a->tokens;
    p.max_tokens = a->max_tokens;
    p.window = a->window;
    p.scale_log2 = a->scale * 1.4426950408889634f;
    p.ctas = pl.ctas;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.prefix = reinterpret_cast<long long *>(ws);
    p.part_ml = reinterpret_cast<float *>(ws + pl.prefix_bytes);
    p.part_o = reinterpret_cast<float *>(ws + pl.prefix_bytes + pl.ml_bytes);
    const int fixed = (D == 64 ? att_fixed_bytes<64>() : att_fixed_bytes<128>()) + (p.batch + 1) * 8 + 128;
    constexpr int kSmem = 227 * 1024;
    p.stages = std::min(ATT_MAXSTAGES, (kSmem - fixed) / (2 * P * D));
    const int smem = fixed + p.stages * 2 * P * D;
    AttFn f = D == 64 ? (P == 32 ? att_kernel<64, 32>(pl.rt) : att_kernel<64, 64>(pl.rt))
                      : (P == 32 ? att_kernel<128, 32>(pl.rt) : att_kernel<128, 64>(pl.rt));
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return serve_cuda_fail(e, "cudaFuncSetAttribute");
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    f<<<pl.ctas, ATT_THREADS, smem, st>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return serve_cuda_fail(e, "attention launch");
    cudaLaunchAttribute dep{};
    dep.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    dep.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(((int64_t)p.tokens * a->q_heads + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = &dep;
    cfg.numAttrs = 1;
    void (*mf)(const AttParams, int) = D == 64 ? (P == 32 ? cache_attend_merge<64, 32> : cache_attend_merge<64, 64>)
                                               : (P == 32 ? cache_attend_merge<128, 32> : cache_attend_merge<128, 64>);
    e = cudaLaunchKernelEx(&cfg, mf, (const AttParams)p, pl.rt);
    return e == cudaSuccess ? MK_OK : serve_cuda_fail(e, "attention merge launch");
}

}  // extern "C"
