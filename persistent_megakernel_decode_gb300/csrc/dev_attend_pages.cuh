// The kernels of the cache attention over pages (attend.cu says what they do and
// why; prefix.cu has another one for the shared pages of large groups).
#pragma once
#include "dev_attend.cuh"

namespace mk {

// Consumer warps of a CTA.  What sequences have behind a shared prefix is short:
// two CTAs of four on an SM have two of those units in work.
__host__ __device__ constexpr int att_warps(AttKind kind) { return kind == ATT_OWN ? 4 : 8; }
// Are the registers shared out by warpgroups?  Tiles of 8 rows by themselves need
// fewer than a thread of 9 warps has; starting the three idle warps of a producer's
// warpgroup costs a short call more than they give (8 sequences of 512-4096, heads of
// 64: 13.4 us, with them 13.6; window and sinks: 12.6 and 12.9).  Taller tiles would
// spill without (36 rows of 128 dims: 27.1 us, without 28.5).
__host__ __device__ constexpr bool att_split(AttKind kind, int rt) { return kind != ATT_PLAIN || rt > 8; }
// + the producer, in a warpgroup of its own where registers are shared out
__host__ __device__ constexpr int att_threads(AttKind kind, int rt) { return (att_warps(kind) + (att_split(kind, rt) ? 4 : 1)) * 32; }
constexpr int ATT_MAXRING = 32;                     // pages in the ring (one producer lane each)

// Tiles of rt rows: 8 NT rows a warp, up to rt / (8 NT) warps side by side
__host__ __device__ constexpr int att_nt(int rt) { return rt == 8 ? 1 : 2; }

template <int RT>
DEV int att_side(int rows) { return att_side_of(RT, rows); }
template <int RT>
DEV long long att_items(const AttParams &p, int cnt, int np) { return att_items_of(p, RT, cnt, np); }

// CTAs that get work: every range is at least one page's items long, so that
// a page begins in each.
DEV int att_used_of(int rt, long long total, int ctas) { return (int)max(1ll, min((long long)ctas, total / att_side_of(rt, rt))); }
template <int RT>
DEV int att_used(long long total, int ctas) { return att_used_of(RT, total, ctas); }

struct AttShared {
    // A unit is a sequence or a group
    long long *prefix;  // [units + 1]: work items before each
    int4 *seq;          // [units]: AttSeq without hi
    AttGroups groups;
    float2 *scale;      // [ring]: (K scale, V scale without the probabilities' 2^14, so that the sums reach as far as
                        // fp32 does), K scale < 0: page not loaded
    uint64_t *full_k, *full_v, *empty_k, *empty_v;
    int *has_k, *has_v; // [ring]: number of the page whose turn the slot's K and V are at
    float *merge;       // [8 warps][8 NT rows][D + 4]
    float *ml;          // [8 warps][8 NT rows][2]
    int *ctrl;          // [0] abort, [1] CTAs that share the work
    unsigned long long *total;  // items of the launch beside this one
    uint8_t *ring;      // [ring][K page, V page]
};

__host__ __device__ constexpr int att_fixed_bytes(int D, int nt, int warps) {
    return warps * 8 * nt * (D + 4) * 4 + warps * 8 * nt * 2 * 4 + ATT_MAXRING * (8 + 32 + 8) + 16;
}
__host__ __device__ constexpr int att_seq_bytes(int units, int ngroups) {
    return units * 16 + (units + 1) * 8 + att_group_bytes(ngroups);
}

template <int D, int NT, int WARPS>
DEV AttShared att_shared(const AttParams &p, int units) {
    AttShared s;
    uint8_t *at = mk_smem;
    s.full_k = reinterpret_cast<uint64_t *>(at);
    s.full_v = s.full_k + ATT_MAXRING;
    s.empty_k = s.full_v + ATT_MAXRING;
    s.empty_v = s.empty_k + ATT_MAXRING;
    at += ATT_MAXRING * 32;
    s.scale = reinterpret_cast<float2 *>(at);
    at += ATT_MAXRING * 8;
    s.has_k = reinterpret_cast<int *>(at);
    s.has_v = s.has_k + ATT_MAXRING;
    at += ATT_MAXRING * 8;
    s.ctrl = reinterpret_cast<int *>(at);
    s.total = reinterpret_cast<unsigned long long *>(at + 8);
    at += 16;
    s.ml = reinterpret_cast<float *>(at);
    at += WARPS * 8 * NT * 2 * 4;
    s.merge = reinterpret_cast<float *>(at);
    at += WARPS * 8 * NT * (D + 4) * 4;
    s.seq = reinterpret_cast<int4 *>(at);
    s.prefix = reinterpret_cast<long long *>(s.seq + units);
    s.groups = att_groups_at(s.prefix + units + 1, p.ngroups);
    const uint32_t used = (uint32_t)(at - mk_smem) + att_seq_bytes(units, p.ngroups);
    s.ring = mk_smem + ((used + 127) & ~127u);
    return s;
}

// The pages of a sequence that the rows of one of its tiles see: [lo, hi), and below hi those of the sinks.
template <int P, int RT>
DEV void att_tile_pages(const AttParams &p, int cnt, int len, int tile, int &lo, int &hi) {
    const int rows = cnt * p.group;
    const int i0 = tile * RT / p.group, i1 = (min((tile + 1) * RT, rows) - 1) / p.group;
    const int top = len - cnt + i1, bottom = len - cnt + i0;
    hi = top < 0 ? 0 : top / P + 1;
    lo = att_least(bottom, p.window) / P;
}

// One range of pages of one unit, as every warp of the CTA walks them.  A page
// belongs to the CTA in whose range its first item lies.
struct AttSeg {
    int b, tile, h, pg, n;    // the pg-th page that the unit's rows see, and the n - 1 next
    int q0, cnt, len, gap;
    bool whole;               // the unit's every page
    bool head;                // the unit's first page among them
};

template <int P, int RT, AttKind KIND>
struct AttWalk {
    const AttParams &p;
    const AttShared &s;
    long long x, end;
    int b;
    DEV AttWalk(const AttParams &p_, const AttShared &s_) : p(p_), s(s_) {
        const int units = att_units(p, KIND);
        const long long total = s.prefix[units];
        const int ctas = att_used<RT>(total, KIND != ATT_PLAIN ? s.ctrl[1] : p.ctas);
        x = end = 0;
        if ((int)blockIdx.x < ctas) {
            x = att_div((long long)blockIdx.x * total, ctas);
            end = att_div((long long)(blockIdx.x + 1) * total, ctas);
        }
        b = att_find(s.prefix, units, x);
    }
    DEV bool next(AttSeg &g) {
        while (x < end) {
            while (s.prefix[b + 1] <= x) ++b;
            const int4 q = s.seq[b];
            const int np = (q.z + P - 1) / P - q.w, rows = q.y * p.group, tiles = (rows + RT - 1) / RT;
            // the full tiles' units, then the last tile's
            constexpr int FULL_SIDE = RT / (8 * att_nt(RT)), FIXED = att_fixed_items(RT);
            long long r = x - s.prefix[b];
            const long long full = (long long)(tiles - 1) * p.c.hkv * (np * FULL_SIDE + FIXED);
            const bool last = r >= full;
            const int side = last ? att_side<RT>(rows - (tiles - 1) * RT) : FULL_SIDE;
            if (last) r -= full;
            const long long items = (long long)np * side + FIXED;
            int unit = (int)att_div(r, items);
            const int within = (int)(r - unit * items);
            if (last) unit += (tiles - 1) * p.c.hkv;
            const long long left = items - within;  // items to the unit's end
            // the first page that begins at or after x, and at or after the range's end
            const int first = max(0, within - FIXED + side - 1) / side;
            const int until = left <= end - x ? np : max(0, within + (int)(end - x) - FIXED + side - 1) / side;
            x += min(left, end - x);
            if (first >= until) continue;
            g.b = b;
            g.tile = unit / p.c.hkv;
            g.h = unit - g.tile * p.c.hkv;
            g.pg = first;
            g.gap = q.w;
            g.n = until - first;
            g.q0 = q.x;
            g.cnt = q.y;
            g.len = q.z;
            g.whole = g.n == np;
            g.head = first == 0;
            return true;
        }
        return false;
    }
};

// Wait until a slot holds page `number`, bounded (a few seconds): false if it
// ran out or another warp gave up.  The barrier's parity alone does not say
// which page landed: a slot's pages belong to different warps, and one that
// is ahead could take the landing before last for its own.
DEV bool att_wait(const AttParams &p, const AttShared &s, int *has, int number, uint64_t *bar, uint32_t parity) {
    bool asked = ld_acquire_cta(has) == number;
    if (asked && mbar_test(bar, parity)) return true;
    for (int i = 0; i < 4000000; ++i) {
        if (!asked) {
            asked = ld_acquire_cta(has) == number;
            if (!asked && i > 1000) __nanosleep(1000);
        } else {
            if (mbar_wait_hint(bar, parity, 100000)) return true;
            i += 1000;
        }
        if (*reinterpret_cast<volatile int *>(s.ctrl)) return false;
    }
    note_failure(p.c.status, MK_ERR_TIMEOUT, -1, blockIdx.x, -1);
    *reinterpret_cast<volatile int *>(s.ctrl) = 1;
    return false;
}

// The producer warp.  Lane i of a batch of `ring` pages looks up and loads the
// i-th: a loop over pages in one thread took 850 clocks a page, all of them
// instruction latency.  All lanes poll their slots at once; those that are
// free are filled.
template <int D, int P, int RT, AttKind KIND>
DEV void att_produce(const AttParams &p, const AttShared &s) {
    constexpr int PAGE = P * D;
    const int lane = threadIdx.x % 32;
    uint8_t *dst = s.ring + (size_t)lane * 2 * PAGE;
    AttWalk<P, RT, KIND> walk(p, s);
    AttSeg g;
    bool more = walk.next(g);
    int before = 0;  // pages of the ranges done
    // The CTA's page number base + lane: this lane's next (want), its number
    // (-1: not loaded) and its kv head.
    const auto look = [&](int base, bool &want, int &id, int &h) {
        want = false;
        id = -1;
        h = 0;
        int b = -1, pg = 0;
        while (more) {
            const int k = base + lane - before;
            if (lane < p.ring && k >= 0 && k < g.n) {
                want = true;
                h = g.h;
                pg = att_page(p, g.pg + k, g.gap);
                if (KIND == ATT_GROUPS) {
                    b = s.groups.lead[g.b];
                } else {
                    int lo, hi;
                    att_tile_pages<P, RT>(p, g.cnt, g.len, g.tile, lo, hi);
                    if ((pg >= lo || pg < p.sink_pages) && pg < hi) b = g.b;
                }
            }
            if (before + g.n >= base + p.ring) break;
            before += g.n;
            more = walk.next(g);
        }
        if (b >= 0) {  // all lanes' table entries at once
            id = p.table[(size_t)b * p.width + pg];
            if ((unsigned)id >= (unsigned)p.c.pages) {
                note_failure(p.c.status, MK_ERR_DEVICE_CHECK, b, pg * P, id);
                id = -1;
            }
        }
    };
    bool want;
    int id, h;
    look(0, want, id, h);
    uint32_t turn = 0, k_fills = 0, v_fills = 0;
    bool ok = true;
    for (; ok && __any_sync(FULL, want); ++turn) {
        const size_t at = (size_t)(id < 0 ? 0 : id) * p.c.hkv + h;
        float2 sc = make_float2(-1.f, 0.f);
        if (id >= 0) sc = make_float2(p.c.ks[at], p.c.vs[at] * 0x1p-14f);
        const int now = id;
        bool k_todo = want, v_todo = want;
        const uint32_t ph = (turn & 1) ^ 1;
        for (int spin = 0; __any_sync(FULL, k_todo || v_todo); ++spin) {
            const bool k = k_todo && (turn == 0 || mbar_test(&s.empty_k[lane], ph));
            if (k && now >= 0) {
                mbar_expect_tx(&s.full_k[lane], PAGE);
                bulk_g2s_plain(dst, p.c.k + at * PAGE, PAGE, &s.full_k[lane]);
            }
            const bool v = v_todo && (turn == 0 || mbar_test(&s.empty_v[lane], ph));
            if (v) st_release_cta(&s.has_v[lane], (int)turn * p.ring + lane);
            if (v && now >= 0) {
                mbar_expect_tx(&s.full_v[lane], PAGE);
                bulk_g2s_plain(dst + PAGE, p.c.v + at * PAGE, PAGE, &s.full_v[lane]);
            }
            if (k) {  // full_k counts two arrivals: the scales come with the second
                s.scale[lane] = sc;
                st_release_cta(&s.has_k[lane], (int)turn * p.ring + lane);
                mbar_arrive(&s.full_k[lane]);
                if (now < 0) mbar_arrive(&s.full_k[lane]);
            }
            if (v && now < 0) mbar_arrive(&s.full_v[lane]);
            k_todo = k_todo && !k;
            v_todo = v_todo && !v;
            k_fills += k;
            v_fills += v;
            if (spin == 0) look(((int)turn + 1) * p.ring, want, id, h);  // the next turn's, while this one's slots come free
            if (spin > 256) {
                __nanosleep(spin > 4096 ? 1000 : 100);
                const bool give_up = spin > 4000000 || *reinterpret_cast<volatile int *>(s.ctrl);  // a few seconds
                if (__any_sync(FULL, give_up)) {
                    ok = false;
                    break;
                }
            }
        }
    }
    if (!ok) {
        if (lane == 0) note_failure(p.c.status, MK_ERR_TIMEOUT, -1, blockIdx.x, -1);
        *reinterpret_cast<volatile int *>(s.ctrl) = 1;
    }
    // the copies in flight land before the CTA ends, also where the warps that wanted them have given up
    for (int i = 0; i < 200 && k_fills && !mbar_wait_hint(&s.full_k[lane], (k_fills - 1) & 1, 1000000); ++i) {
    }
    for (int i = 0; i < 200 && v_fills && !mbar_wait_hint(&s.full_v[lane], (v_fills - 1) & 1, 1000000); ++i) {
    }
}

DEV void att_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit values, two a thread (row lane / 4), transposed.
DEV uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Bytes of w that are e4m3's NaN codes (0x7f, 0xff), as a byte mask.
DEV uint32_t nan_bytes(uint32_t w) {
    const uint32_t m = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
    return m * 0xffu;
}

// One row of the query operand: f16 pairs of dims h2 * 64 + 16 t .. + 15;
// returns 2^-k of the row's scaling (NaN if the row is not finite).
template <int D>
DEV float att_load_q(const uint16_t *row, int t, uint32_t (&qb)[D / 64][8]) {
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
    // times 2^(14 - exponent) (bits 127 + 14 - (field - 127)): the row's largest value lands in [2^14, 2^15)
    const int up = min(max(268 - (int)(big >> 23), 1), 253);
    const float sc = __uint_as_float((uint32_t)up << 23);
#pragma unroll
    for (int h2 = 0; h2 < D / 64; ++h2)
#pragma unroll
        for (int i = 0; i < 8; ++i) qb[h2][i] = half2_of(f[h2][2 * i] * sc, f[h2][2 * i + 1] * sc);
    return big >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(254 - up) << 23);
}

// n arrivals at once
DEV void mbar_arrive_n(uint64_t *b, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(saddr(b)), "r"(n) : "memory");
}
// This thread's loads from shared memory come before copies that another thread
// starts after an arrival behind this.  Copies are the async proxy's, loads the
// generic one's: an arrival alone does not order them.  Without it a slot's next
// page landed under the last loads once in some 10,000 calls with pages of 32 tokens
// and heads of 128, whose rows conflict eight ways and wait longest in the load
// queue.  (36 rows of 128 dims: 26.9 us, without 26.6; releasing K behind the
// maxima instead, which need all of it, 27.2.)
DEV void att_reads_done() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
template <int WARPS>
DEV void att_consumer_bar() { asm volatile("bar.sync 1, %0;" ::"n"(WARPS * 32) : "memory"); }

template <int D, int P, int RT, AttKind KIND>
DEV void att_consume(const AttParams &p, const AttShared &s) {
    constexpr int WARPS = att_warps(KIND), NT = att_nt(RT), WT = RT / (8 * NT);  // 8-row tiles a warp, warps for a full tile
    constexpr int PAGE = P * D, RUN = P / 4, NM = P / 16, ND = D / 16, LD = D + 4;
    constexpr bool QS = NT > 1;  // the query operand in shared memory (registers would spill)
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g8 = lane / 4, t = lane % 4;
    AttWalk<P, RT, KIND> walk(p, s);
    AttSeg g;
    bool ok = true;
    int before = 0;  // pages of the CTA's ranges done
    while (walk.next(g)) {
        constexpr bool all = KIND == ATT_GROUPS;  // every row sees every token
        const int rows = g.cnt * p.group, base = all ? g.len - 1 : g.len - g.cnt;
        // as many warps side by side as the tile's rows need (1, 2 or 4), the
        // others on other pages: group grp takes every ng-th page of the range
        const int side = att_side<RT>(rows - g.tile * RT);
        const int wt = warp % side, grp = warp / side, ng = WARPS / side;
        const int row0 = g.tile * RT + wt * 8 * NT;
        int st = (before + grp) % p.ring;  // ring slot and phase of this warp's next page
        uint32_t ph = ((before + grp) / p.ring) & 1;
        const auto settle = [&] {
            while (st >= p.ring) {
                st -= p.ring;
                ph ^= 1;
            }
        };
        const auto pos_of = [&](int r) {  // a row sees [least, pos], and below it the sinks
            return r < rows ? base + (all ? 0 : r / p.group) : -1;
        };
        const auto least_of = [&](int pos) { return att_least(pos, p.window); };
        uint32_t qb[QS ? 1 : NT][D / 64][8];
        // fragment j of tile n: qs[((n * D / 64 + h2) * 2 + j) * 32 + lane]
        uint4 *qs = reinterpret_cast<uint4 *>(s.merge) + wt * (NT * D / 32) * 32;
        float f[NT][2], m[NT][2], l[NT][2], o[NT][ND][4];
        int pos[NT][2];
        int all_hi = INT_MAX, all_lo = 0;  // pages within need no masks
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int r = row0 + 8 * n + g8;  // this thread's row of the operand
            const uint16_t *qrow = nullptr;
            if (r < rows) {
                const int tok = r / p.group;
                qrow = p.q + (int64_t)(g.q0 + tok) * p.qs_t + (int64_t)(g.h * p.group + r - tok * p.group) * p.qs_h;
                all_hi = min(all_hi, pos_of(r));
                all_lo = max(all_lo, least_of(pos_of(r)));
            }
            const float qf = att_load_q<D>(qrow, t, qb[QS ? 0 : n]) * p.scale_log2;
            if constexpr (QS)
                if (grp == 0)
#pragma unroll
                    for (int i = 0; i < D / 32; ++i)
                        qs[(n * (D / 32) + i) * 32 + lane] = make_uint4(qb[0][i / 2][4 * (i % 2)], qb[0][i / 2][4 * (i % 2) + 1],
                                                                        qb[0][i / 2][4 * (i % 2) + 2], qb[0][i / 2][4 * (i % 2) + 3]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // its columns of the products
                f[n][e] = __shfl_sync(FULL, qf, 8 * t + 4 * e);
                pos[n][e] = pos_of(row0 + 8 * n + 2 * t + e);
                m[n][e] = -INFINITY;
                l[n][e] = 0.f;
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) o[n][d][0] = o[n][d][1] = o[n][d][2] = o[n][d][3] = 0.f;
        }
        all_hi = __reduce_min_sync(FULL, all_hi);
        all_lo = __reduce_max_sync(FULL, all_lo);
        if constexpr (QS) att_consumer_bar<WARPS>();
        for (int mine = before + grp; mine < before + g.n; mine += ng, st += ng, settle()) {
            const int pg = att_page(p, g.pg + mine - before, g.gap);
            if (ok) ok = att_wait(p, s, &s.has_k[st], mine, &s.full_k[st], ph);
            ok = __all_sync(FULL, ok);
            if (!ok) continue;
            const float2 sc = s.scale[st];
            const bool there = sc.x >= 0.f || sc.x != sc.x;
            const uint8_t *kp = s.ring + (size_t)st * 2 * PAGE, *vp = kp + PAGE;
            if (there) {
                const bool edge = (pg * P < all_lo && pg * P + P - 1 >= p.sinks) || pg * P + P - 1 > all_hi;
                float c[NT][NM][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < NM; ++i) c[n][i][0] = c[n][i][1] = c[n][i][2] = c[n][i][3] = 0.f;
                const uint8_t *kr = kp + (RUN * (g8 >> 1) + (g8 & 1)) * D + 16 * t;
                // 32 dims at a time, so that consecutive products go to different sums
#pragma unroll
                for (int h2 = 0; h2 < D / 64; ++h2)
#pragma unroll
                    for (int jj = 0; jj < 2; ++jj) {
                        uint2 x[NM], y[NM];
#pragma unroll
                        for (int i = 0; i < NM; ++i) {
                            x[i] = *reinterpret_cast<const uint2 *>(kr + 4 * i * D + h2 * 64 + 8 * jj);
                            y[i] = *reinterpret_cast<const uint2 *>(kr + (4 * i + 2) * D + h2 * 64 + 8 * jj);
                        }
                        uint4 qj[NT];
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            if constexpr (QS) qj[n] = qs[(n * (D / 32) + 2 * h2 + jj) * 32 + lane];
                            else qj[n] = make_uint4(qb[n][h2][4 * jj], qb[n][h2][4 * jj + 1], qb[n][h2][4 * jj + 2], qb[n][h2][4 * jj + 3]);
                        }
#pragma unroll
                        for (int j = 0; j < 2; ++j)
#pragma unroll
                            for (int i = 0; i < NM; ++i) {
                                const uint32_t xw = j ? x[i].y : x[i].x, yw = j ? y[i].y : y[i].x;
                                uint32_t a0, a1, a2, a3;
                                e4m3x4_to_half2(xw, a0, a2);
                                e4m3x4_to_half2(yw, a1, a3);
#pragma unroll
                                for (int n = 0; n < NT; ++n)
                                    att_mma(c[n][i], a0, a1, a2, a3, j ? qj[n].z : qj[n].x, j ? qj[n].w : qj[n].y);
                            }
                    }
                att_reads_done();
                __syncwarp();
                if (lane == 0) mbar_arrive_n(&s.empty_k[st], WT / side);  // K is read: the next one loads during the rest
                const int first = pg * P + RUN * (g8 >> 1) + (g8 & 1);  // token of c[.][0][0]; [i][2u + e]: + 4 i + 2 u
                float alpha[NT][2];
                uint32_t pb[NT][NM][2];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float fk = f[n][e] * sc.x;
#pragma unroll
                        for (int i = 0; i < NM; ++i)
#pragma unroll
                            for (int u = 0; u < 2; ++u) c[n][i][2 * u + e] *= fk;
                    }
                if (__builtin_expect(edge, 0)) {
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int least = least_of(pos[n][e]);
#pragma unroll
                            for (int i = 0; i < NM; ++i)
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    const int x = first + 4 * i + 2 * u;
                                    if (x > pos[n][e] || (x < least && x >= p.sinks)) c[n][i][2 * u + e] = -INFINITY;
                                }
                        }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float mx = fmaxf(c[n][0][e], c[n][0][2 + e]);
#pragma unroll
                        for (int i = 1; i < NM; ++i) mx = fmaxf(mx, fmaxf(c[n][i][e], c[n][i][2 + e]));
                        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, 16));
                        const float mn = fmaxf(m[n][e], mx), mu = mn == -INFINITY ? 0.f : mn;
                        alpha[n][e] = exp2_fast(m[n][e] - mu);
                        m[n][e] = mn;
                        float sum = 0.f;
#pragma unroll
                        for (int i = 0; i < NM; ++i)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const float x = exp2_fast(c[n][i][2 * u + e] - mu + 14.f);
                                c[n][i][2 * u + e] = x;
                                sum += x;
                            }
                        l[n][e] = fmaf(l[n][e], alpha[n][e], sum);
                    }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < NM; ++i)
#pragma unroll
                        for (int u = 0; u < 2; ++u) pb[n][i][u] = transpose8(half2_of(c[n][i][2 * u], c[n][i][2 * u + 1]));
                ok = att_wait(p, s, &s.has_v[st], mine, &s.full_v[st], ph);
                ok = __all_sync(FULL, ok);
                // A masked token's weight is 0, but 0 x NaN is NaN: where masks
                // apply, NaN codes are taken out, and a product of the mask with
                // their places says which sums really contain one.
                bool dirty = false;
                if (__builtin_expect(edge, 0)) {
                    uint32_t bad = 0;
#pragma unroll 1
                    for (int i = lane; i < PAGE / 16; i += 32) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(vp + 16 * i);
                        bad |= nan_bytes(x.x) | nan_bytes(x.y) | nan_bytes(x.z) | nan_bytes(x.w);
                    }
                    dirty = __any_sync(FULL, bad != 0);
                }
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    uint32_t w[2][RUN / 4];
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint8_t *vr = vp + (d * 16 + 8 * u + g8) * P + RUN * t;
                        if constexpr (P == 64) {
                            const uint4 x = *reinterpret_cast<const uint4 *>(vr);
                            w[u][0] = x.x, w[u][1] = x.y, w[u][2] = x.z, w[u][3] = x.w;
                        } else {
                            const uint2 x = *reinterpret_cast<const uint2 *>(vr);
                            w[u][0] = x.x, w[u][1] = x.y;
                        }
                    }
                    if (__builtin_expect(dirty, 0)) {
                        uint32_t at[2][RUN / 4];
#pragma unroll
                        for (int i = 0; i < RUN / 4; ++i)
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const uint32_t nb = nan_bytes(w[u][i]);
                                w[u][i] &= ~nb;
                                at[u][i] = nb & 0x38383838u;  // 1.0
                            }
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const int ps = pos_of(row0 + 8 * n + g8), ls = least_of(ps);
                            float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                            for (int i = 0; i < RUN / 4; ++i) {
                                uint32_t see[2];
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const int x = pg * P + RUN * t + 4 * i + 2 * k;
                                    see[k] = (x <= ps && (x >= ls || x < p.sinks) ? 0x3c00u : 0u) |
                                             (x + 1 <= ps && (x + 1 >= ls || x + 1 < p.sinks) ? 0x3c000000u : 0u);
                                }
                                att_mma(z, e4m3x2_to_half2(at[0][i]), e4m3x2_to_half2(at[1][i]),
                                        e4m3x2_to_half2(at[0][i] >> 16), e4m3x2_to_half2(at[1][i] >> 16), see[0], see[1]);
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                if (z[k] > 0.f) o[n][d][k] = __uint_as_float(0x7fc00000u);
                        }
                    }
                    float a[NT][4];
#pragma unroll
                    for (int n = 0; n < NT; ++n) a[n][0] = a[n][1] = a[n][2] = a[n][3] = 0.f;
#pragma unroll
                    for (int i = 0; i < RUN / 4; ++i) {
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_to_half2(w[0][i], a0, a2);
                        e4m3x4_to_half2(w[1][i], a1, a3);
#pragma unroll
                        for (int n = 0; n < NT; ++n) att_mma(a[n], a0, a1, a2, a3, pb[n][i][0], pb[n][i][1]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int k = 0; k < 4; ++k) o[n][d][k] = fmaf(a[n][k], sc.y, o[n][d][k] * alpha[n][k % 2]);
                }
            }
            if (!there) {
                // Not loaded, but its V has a turn too: warps of the page before it
                // may still read the slot's V, and arriving now would be taken for them.
                __syncwarp();
                if (lane == 0) mbar_arrive_n(&s.empty_k[st], WT / side);
                ok = att_wait(p, s, &s.has_v[st], mine, &s.full_v[st], ph);
                ok = __all_sync(FULL, ok);
            }
            att_reads_done();
            __syncwarp();
            if (ok && lane == 0) mbar_arrive_n(&s.empty_v[st], WT / side);
        }
        before += g.n;
        // merge the ng warps of each tile
        if constexpr (QS) att_consumer_bar<WARPS>();  // the query operand lies where the sums go
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float *mo = s.merge + ((warp * NT + n) * 8 + 2 * t) * LD + g8;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[n][e];
                sum += __shfl_xor_sync(FULL, sum, 4);
                sum += __shfl_xor_sync(FULL, sum, 8);
                sum += __shfl_xor_sync(FULL, sum, 16);
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    mo[e * LD + 16 * d] = o[n][d][e];
                    mo[e * LD + 16 * d + 8] = o[n][d][2 + e];
                }
                if (g8 == 0) *reinterpret_cast<float2 *>(s.ml + ((warp * NT + n) * 8 + 2 * t + e) * 2) = make_float2(m[n][e], sum);
            }
        }
        att_consumer_bar<WARPS>();
        for (int i = threadIdx.x; i < RT * (D / 4); i += WARPS * 32) {
            const int row = i / (D / 4), d4 = i % (D / 4);
            const int rr = g.tile * RT + row;
            if (rr >= rows) continue;
            // row of the tile -> (warp side by side, row of the warp); group k is `side` warps further
            const auto at = [&](int k) { return (k * side + row / (8 * NT)) * 8 * NT + row % (8 * NT); };
            float big = -INFINITY;
            for (int k = 0; k < ng; ++k) big = fmaxf(big, s.ml[at(k) * 2]);
            const float mu = big == -INFINITY ? 0.f : big;
            float sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int k = 0; k < ng; ++k) {
                const float a = exp2_fast(s.ml[at(k) * 2] - mu);
                const float4 x = *reinterpret_cast<const float4 *>(s.merge + at(k) * LD + 4 * d4);
                sum = fmaf(a, s.ml[at(k) * 2 + 1], sum);
                acc.x = fmaf(a, x.x, acc.x);
                acc.y = fmaf(a, x.y, acc.y);
                acc.z = fmaf(a, x.z, acc.z);
                acc.w = fmaf(a, x.w, acc.w);
            }
            if (KIND != ATT_PLAIN && g.whole) {
                const size_t at_row = (((size_t)all * p.tokens + g.q0 + rr / p.group) * p.c.hkv + g.h) * p.group + rr % p.group;
                *reinterpret_cast<float4 *>(p.row_o + at_row * D + 4 * d4) = acc;
                if (d4 == 0) *reinterpret_cast<float2 *>(p.row_ml + at_row * 2) = make_float2(big, sum);
            } else if (g.whole) {
                const int64_t token = g.q0 + rr / p.group;
                const int hd = g.h * p.group + rr % p.group;
                const float inv = att_inverse(sum);
                *reinterpret_cast<uint2 *>(p.out + token * p.os_t + (int64_t)hd * p.os_h + 4 * d4) =
                    make_uint2(bf16_pair(acc.x * inv, acc.y * inv), bf16_pair(acc.z * inv, acc.w * inv));
                if (p.lse && d4 == 0)
                    p.lse[token * (p.group * p.c.hkv) + hd] = att_lse(big, sum);
            } else {
                const size_t slot = ((size_t)blockIdx.x * 2 + (g.head ? 1 : 0)) * RT + row;
                *reinterpret_cast<float4 *>((all ? p.pre_o : p.part_o) + slot * D + 4 * d4) = acc;
                if (d4 == 0) *reinterpret_cast<float2 *>((all ? p.pre_ml : p.part_ml) + slot * 2) = make_float2(big, sum);
            }
        }
        att_consumer_bar<WARPS>();
    }
}

template <int D, int P, int RT, AttKind KIND>
__global__ void __launch_bounds__(att_threads(KIND, RT), KIND == ATT_OWN ? 2 : 1) cache_attend_kernel(const AttParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int WARPS = att_warps(KIND), THREADS = att_threads(KIND, RT);
    const AttShared s = att_shared<D, att_nt(RT), WARPS>(p, att_units(p, KIND));
    const int tid = threadIdx.x, units = att_units(p, KIND);
    AttSeq seq{0, 0, 0, 0, 0, false};
    if constexpr (KIND != ATT_PLAIN) seq = att_groups<P>(p, s.groups, KIND == ATT_OWN && blockIdx.x == 0);
    for (int b = tid; b < units; b += THREADS) {
        const AttSeq q = att_unit<P, KIND>(p, s.groups, b, KIND != ATT_GROUPS && blockIdx.x == 0, &seq);
        s.prefix[b + 1] = att_items<RT>(p, q.cnt, q.hi - q.gap);
        s.seq[b] = make_int4(q.q0, q.cnt, q.len, q.gap);
    }
    if (tid >= THREADS - 32 && tid - (THREADS - 32) < p.ring) {
        const int i = tid - (THREADS - 32);
        s.has_k[i] = s.has_v[i] = -1;
        mbar_init(&s.full_k[i], 2);
        mbar_init(&s.full_v[i], 1);
        mbar_init(&s.empty_k[i], RT / (8 * att_nt(RT)));
        mbar_init(&s.empty_v[i], RT / (8 * att_nt(RT)));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) s.ctrl[0] = 0, *s.total = 0;
    att_running(s.prefix, units);
    if constexpr (KIND != ATT_PLAIN) {
        att_others<P, KIND>(p, s.groups, seq, s.total);
        __syncthreads();
        const long long mine = s.prefix[units], others = (long long)*s.total;
        const int share = KIND == ATT_GROUPS ? att_share(p, mine, others) : 2 * (p.sms - att_share(p, others, mine));
        if (tid == 0) s.ctrl[1] = min(p.ctas, share);
        __syncthreads();
        // (one CTA at least of the second of both: it ends after the first)
        if ((int)blockIdx.x >= max(s.ctrl[1], KIND == ATT_OWN ? 1 : 0)) return;
    }
    // Registers: 3 x 128 threads were launched with 168 each (an SM's quarter holds
    // three warps of that size): 2 x 216 + 72; twice 2 x 128 with 128: 184 + 72.
    // What does not fit goes to local memory, for which shared memory leaves hardly
    // any L1 cache.
    if (tid >= WARPS * 32) {
        if constexpr (att_split(KIND, RT)) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (tid < (WARPS + 1) * 32) att_produce<D, P, RT, KIND>(p, s);
    } else {
        if constexpr (KIND == ATT_OWN) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        else if constexpr (att_split(KIND, RT)) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        att_consume<D, P, RT, KIND>(p, s);
    }
    // the groups' launch, beside which this one ran, is done before this one is
    if constexpr (KIND == ATT_OWN)
        if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// One warp per query row: rows that see nothing get zeros, rows whose pages
// two or more CTAs shared are merged, in the order of the CTAs; the others
// are written already.  With shared prefixes all rows are merged, the own
// tokens' part first.  All that does not need the main kernel's results (the
// sequences' running page counts again, the row's sequence) runs while that
// one still does.
template <int D, int P, int RT, AttKind KIND>
__global__ void __launch_bounds__(256) cache_attend_merge(const AttParams p) {
    long long *prefix = reinterpret_cast<long long *>(mk_smem);
    const int tid = threadIdx.x, lane = tid % 32, heads = p.group * p.c.hkv, units = p.batch;
    constexpr bool SH = KIND != ATT_PLAIN;
    const AttGroups groups = att_groups_at(prefix + units + 1, p.ngroups);
    AttSeq seq{0, 0, 0, 0, 0, false};
    if constexpr (SH) seq = att_groups<P>(p, groups, false);
    for (int b = tid; b < units; b += 256) {
        const AttSeq q = att_unit<P, KIND>(p, groups, b, false, &seq);
        prefix[b + 1] = att_items<RT>(p, q.cnt, q.hi - q.gap);
    }
    att_running(prefix, units);
    // items of the groups' launch
    long long *before = reinterpret_cast<long long *>(mk_smem + (units + 1) * 8 + (att_group_bytes(p.ngroups) + 7) / 8 * 8);
    if constexpr (SH) {
        for (int g = tid; g < p.ngroups; g += 256) {
            const AttSeq q = att_unit<P, ATT_GROUPS>(p, groups, g, false);
            before[g + 1] = att_group_items(p, q.cnt, q.hi);
        }
        att_running(before, p.ngroups);
    }
    const int64_t w = (int64_t)blockIdx.x * 8 + tid / 32;
    const int token = (int)min(w / heads, (int64_t)p.tokens - 1), head = (int)(w % heads);
    int b = 0;
    if (p.q_start) {
        int z = p.batch;  // the last b with q_start[b] <= token
        while (z - b > 1) {
            const int mid = (b + z) / 2;
            if (p.q_start[mid] <= token) b = mid;
            else z = mid;
        }
    } else {
        b = min(token / p.max_tokens, p.batch - 1);
    }
    // the CTAs that have parts of the row in one unit (n pages; c0 > c1: one
    // CTA had it all), and the row's place in its tile
    struct Part {
        int n, c0, c1, row;
    };
    const long long total = prefix[units];
    const int pre_ctas = SH ? att_share(p, before[p.ngroups], total) : 0;
    const int ctas = att_used<RT>(total, SH ? min(p.ctas, 2 * (p.sms - pre_ctas)) : p.ctas);
    // of tiles of rt rows, a unit's first item being number `first`
    const auto part_of = [&](const AttSeq &s, int rt, long long first, long long all, int n, bool whole_pages) {
        Part x{s.hi - s.gap, 0, -1, 0};
        if (x.n <= 0 || s.cnt <= 0) {
            x.n = 0;
            return x;
        }
        const int h = head / p.group, r = (token - s.q0) * p.group + head % p.group;
        const int rows = s.cnt * p.group, tile = r / rt;
        const int side = whole_pages ? 1 : att_side_of(rt, rows - tile * rt), full = whole_pages ? 1 : att_side_of(rt, rt);
        const int fixed = whole_pages ? PRE_FIXED : att_fixed_items(rt);
        const long long x0 = first + (long long)tile * p.c.hkv * ((long long)x.n * full + fixed) +
                             h * ((long long)x.n * side + fixed) + fixed;  // the first page's item
        const int c0 = att_owner(x0, all, n), c1 = att_owner(x0 + (long long)(x.n - 1) * side, all, n);
        if (c0 != c1) {
            x.c0 = c0;
            x.c1 = c1;
        }
        x.row = r % rt;
        return x;
    };
    const AttSeq s = att_unit<P, KIND>(p, groups, b, false);
    bool todo = w < (int64_t)p.tokens * heads && token >= s.q0 && token < s.q0 + s.cnt;
    Part own{0, 0, -1, 0}, pre{0, 0, -1, 0};
    if (todo) {
        own = part_of(s, RT, prefix[b], total, ctas, false);
        if constexpr (SH) {
            const int g = att_group_of(p, groups, b);
            if (g >= 0) {
                const bool whole_pages = p.pre_rt == PRE_ROWS;
                const long long all = before[p.ngroups];
                pre = part_of(att_unit<P, ATT_GROUPS>(p, groups, g, false), p.pre_rt, before[g], all,
                              whole_pages ? pre_used(all, pre_ctas) : att_used_of(p.pre_rt, all, min(p.sms, pre_ctas)), whole_pages);
            }
        } else {
            todo = own.n == 0 || own.c0 <= own.c1;
        }
    }
    // every thread waits: this grid must not be done before the main kernel is
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!todo) return;
    constexpr int V = D / 32;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    float big = -INFINITY, sum = 0.f;
    // part i of the row: the own tokens' in the order of the CTAs, then the group's
    const int n_own = own.n == 0 ? 0 : own.c0 <= own.c1 ? own.c1 - own.c0 + 1 : SH ? 1 : 0;
    const int n_pre = pre.n == 0 ? 0 : pre.c0 <= pre.c1 ? pre.c1 - pre.c0 + 1 : 1;
    const auto at = [&](int i, const float *&ml, const float *&o) {
        const bool shared = SH && i >= n_own;
        const Part &x = shared ? pre : own;
        if (shared) i -= n_own;
        if (SH && x.c0 > x.c1) {  // one CTA had it all
            const size_t row = ((size_t)shared * p.tokens + token) * heads + head;
            ml = p.row_ml + row * 2;
            o = p.row_o + row * D;
            return;
        }
        const size_t slot = ((size_t)(x.c0 + i) * 2 + (i == 0 ? 1 : 0)) * (shared ? p.pre_rt : RT) + x.row;  // c0 has the unit's head
        ml = (shared ? p.pre_ml : p.part_ml) + slot * 2;
        o = (shared ? p.pre_o : p.part_o) + slot * D;
    };
    for (int c = 0; c < n_own + n_pre; c += 32) {  // the maxima first, 32 parts at a time
        const int n = min(32, n_own + n_pre - c);
        const float *ml_at, *o_at = nullptr;
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < n) {
            at(c + lane, ml_at, o_at);
            ml = *reinterpret_cast<const float2 *>(ml_at);
        }
        const float top = fmaxf(big, warp_max(ml.x)), mu = top == -INFINITY ? 0.f : top;
        const float a = exp2_fast(big - mu), e = exp2_fast(ml.x - mu);
        big = top;
        sum *= a;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= a;
#pragma unroll 8
        for (int j = 0; j < n; ++j) {
            const float ej = __shfl_sync(FULL, e, j), lj = __shfl_sync(FULL, ml.y, j);
            const float *o = reinterpret_cast<const float *>(__shfl_sync(FULL, reinterpret_cast<unsigned long long>(o_at), j)) + lane * V;
            sum = fmaf(lj, ej, sum);
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(o[i], ej, acc[i]);
        }
    }
    const float inv = att_inverse(sum);
    uint16_t *dst = p.out + (int64_t)token * p.os_t + (int64_t)head * p.os_h + lane * V;
#pragma unroll
    for (int i = 0; i < V; i += 2) *reinterpret_cast<uint32_t *>(dst + i) = bf16_pair(acc[i] * inv, acc[i + 1] * inv);
    if (p.lse && lane == 0) p.lse[w] = att_lse(big, sum);
}

using AttFn = void (*)(const AttParams);
template <int D, int P, AttKind KIND>
static AttFn att_kernel(int rt) {
    return rt == 8 ? cache_attend_kernel<D, P, 8, KIND> : rt == 16 ? cache_attend_kernel<D, P, 16, KIND>
         : rt == 32 ? cache_attend_kernel<D, P, 32, KIND> : cache_attend_kernel<D, P, 64, KIND>;
}
template <int D, int P, AttKind KIND>
static AttFn att_merge_kernel(int rt) {
    return rt == 8 ? cache_attend_merge<D, P, 8, KIND> : rt == 16 ? cache_attend_merge<D, P, 16, KIND>
         : rt == 32 ? cache_attend_merge<D, P, 32, KIND> : cache_attend_merge<D, P, 64, KIND>;
}
template <AttKind KIND>
static AttFn att_kernel_of(int D, int P, int rt) {
    return D == 64 ? (P == 32 ? att_kernel<64, 32, KIND>(rt) : att_kernel<64, 64, KIND>(rt))
                   : (P == 32 ? att_kernel<128, 32, KIND>(rt) : att_kernel<128, 64, KIND>(rt));
}
template <AttKind KIND>
static AttFn att_merge_of(int D, int P, int rt) {
    return D == 64 ? (P == 32 ? att_merge_kernel<64, 32, KIND>(rt) : att_merge_kernel<64, 64, KIND>(rt))
                   : (P == 32 ? att_merge_kernel<128, 32, KIND>(rt) : att_merge_kernel<128, 64, KIND>(rt));
}
// The shared forms are compiled by themselves (shared.cu).
AttFn att_shared_kernel(AttKind kind, int D, int P, int rt);
AttFn att_shared_merge(int D, int P, int rt);

}  // namespace mk
