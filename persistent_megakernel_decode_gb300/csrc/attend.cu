// Attention of new tokens over an 8-bit paged KV cache.
//
// Mathematics.  One pass over a sequence's pages with the running maximum m
// and sum l of the softmax (in log2 units); partial results of page ranges
// merge as sum_i 2^(m_i - M) (l_i, O_i).  All sums are fp32.
//
// What bounds it: the cache's bytes, 2 D per token and kv head, each read
// once; a group of q heads (and of new tokens) shares them.
//
// Matrix products.  mma.sync m16n8k16 in f16 with fp32 sums, the cache as the
// 16-row operand: scores are K q^T (16 tokens x 8 query rows), outputs V^T
// p^T (16 dims x 8 rows), so that the 8 rows of a decode step's kv head (q
// heads, then new tokens) fill the tile.  Codes become f16 in registers
// (exact).  A query row is scaled by a power of two into f16's range, which
// holds bf16's 8 bits exactly; probabilities are f16 times 2^14, 2^-11 of
// their value.  The other form tried, m16n8k32 on the e4m3 codes themselves
// (each row split into two e4m3 halves at scales 1 and 1/16, one in row g and
// one in row g + 8), needs no conversion in the source but executed 1460
// instructions a page and warp against about 1000 here, and is less exact
// (2^-8).  tcgen05 is not used: its tiles take 64 rows or more of an operand
// from shared memory, a decode step has 4 to 16, and scores would cross tensor
// memory between the two products; bytes bound a decode step either way.
//
// Token order.  A contraction may run over tokens in any order, so row (m, u,
// g) of the score tile (16-row step m, half u, row g) is token (P/4)(g/2) + 4m
// + 2u + g%2 of the page: after an 8 x 8 transpose in registers (movmatrix),
// thread t of a quad holds the probabilities of the P/4 tokens from (P/4) t
// on, and its V operand is one P/4-byte run of a transposed V row.
//
// Work split.  The pages of all units (sequence, row tile, kv head) form one
// axis, each weighted with the warps its tile occupies side by side, and with
// a constant for beginning and merging a unit, cut into equal ranges, one per
// CTA (one CTA per SM): ragged batches and single long sequences balance alike.  A producer warp streams the pages through a
// shared-memory ring with bulk copies; the consumer warps take them in turn
// (as many side by side as the tile's rows need) and merge in shared memory.
// A page that a tile does not see, or whose number is out of range, takes its
// turn in the ring without being loaded.
// A unit that one CTA covers is written at once; ranges cut by a CTA boundary
// go to the workspace and a second small launch (dependent launch, so that its
// start overlaps) merges them in order: results do not depend on timing.
//
// Measured (one GB300, device time): 16 sequences of 16-32K tokens, 32 q / 8
// kv heads of 128: 128 us, 6.1 TB/s, 90 % of the copy rate; 8 sequences of
// 512-4096, heads of 64: 13.0 us, of which the bytes are 2.8
// (two launches, two dependent look-ups, the ramp of the loads and the merge
// are the rest); 64 new tokens a sequence over 4000: 190 TFLOP/s, bound by the
// instructions per product that a 16-row operand held in registers costs; a
// prompt of 2048 new tokens: 377 us, 91 TFLOP/s, half of its tiles' pages
// passing through the ring unseen.
#include <algorithm>
#include <climits>

#include "dev_serve.cuh"

namespace mk {

constexpr int ATT_WARPS = 8;                        // consumer warps
constexpr int ATT_THREADS = (ATT_WARPS + 1) * 32;   // + the producer
constexpr int ATT_MAXB = 1024;                      // sequences per call
constexpr int ATT_MAXRING = 32;                     // pages in the ring (one producer lane each)

struct AttParams {
    CacheView c;  // of the layer: k, v, ks, vs point at it
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    int64_t qs_t, qs_h, os_t, os_h;
    const int *table, *lens, *q_start;
    int batch, width, group, tokens, max_tokens, window, ring, ctas;
    float scale_log2;
    // workspace: partial (m, l) [ctas][2][RT][2]; partial O [ctas][2][RT][D]
    float *part_ml, *part_o;
};

// ln of the sum of exponentials: maximum in log2 units, sum times 2^14.
DEV float att_lse(float big, float sum) {
    return sum == 0.f ? -INFINITY : (big - 14.f + log2f(sum)) * 0.6931471805599453f;
}
// 1 / the sum of exponentials, from their sum times 2^14.
DEV float att_inverse(float sum) { return sum == 0.f ? 0.f : 16384.f / sum; }

// The first position that a query at pos sees (pos < 0: sees none, any window's end fits 32 bits).
DEV int att_least(int pos, int window) { return window > 0 && pos >= window ? pos - window + 1 : 0; }

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

// Tiles of rt rows: 8 NT rows a warp, up to rt / (8 NT) warps side by side
__host__ __device__ constexpr int att_nt(int rt) { return rt == 8 ? 1 : 2; }

// Warps side by side on a tile of so many rows: 1, 2 or 4.
template <int RT>
DEV int att_side(int rows) {
    const int need = (min(RT, rows) + 8 * att_nt(RT) - 1) / (8 * att_nt(RT));
    return need <= 1 ? 1 : need == 2 ? 2 : 4;
}
// What beginning and merging a unit costs a CTA, in items.  By the clock 4 to 5
// thousand clocks, at 375 to 700 an item, with one tile a warp; 10 thousand, at
// 525, with two.  Measured over six sets of lengths, 8 sequences of the 1B
// shape / 13 with up to 9 drafted tokens: none 15.8 / 41 us, 4 and 8 items
// 14.3 / 30, 12 and 24 13.3 / 26.6, 16 and 40 12.7 / 27.3.
__host__ __device__ constexpr int att_fixed_items(int rt) { return rt == 8 ? 12 : 24; }
// Work items of a sequence: of each unit the fixed ones, then its pages', each
// as many as its tile has warps side by side.  All tiles but the last are full.
template <int RT>
DEV long long att_items(const AttParams &p, int cnt, int np) {
    const int rows = cnt * p.group, tiles = (rows + RT - 1) / RT;
    if (tiles == 0 || np == 0) return 0;
    constexpr int FIXED = att_fixed_items(RT);
    return p.c.hkv * ((tiles - 1) * ((long long)np * att_side<RT>(RT) + FIXED) +
                      (long long)np * att_side<RT>(rows - (tiles - 1) * RT) + FIXED);
}
// prefix[1 .. n]: values -> running sums, by the whole block; prefix[0] = 0.
DEV void att_running(long long *prefix, int n) {
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        long long carry = 0;
        if (lane == 0) prefix[0] = 0;
        for (int b0 = 0; b0 < n; b0 += 32) {
            const int b = b0 + lane;
            long long v = b < n ? prefix[b + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long u = __shfl_up_sync(FULL, v, o);
                if (lane >= o) v += u;
            }
            v += carry;
            if (b < n) prefix[b + 1] = v;
            carry = __shfl_sync(FULL, v, 31);
        }
    }
    __syncthreads();
}

// A quotient that mostly fits 32 bits.
DEV long long att_div(long long a, long long b) {
    return (a | b) <= 0xffffffffll ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// CTAs that get work: every range is at least one page's items long, so that
// a page begins in each.
template <int RT>
DEV int att_used(long long total, int ctas) {
    return (int)max(1ll, min((long long)ctas, total / (RT / (8 * att_nt(RT)))));
}
// CTA of work item x when `total` items are cut into `ctas` <= total ranges [c total / ctas, (c + 1) total / ctas).
DEV int att_owner(long long x, long long total, int ctas) { return (int)att_div((x + 1) * ctas - 1, total); }

struct AttShared {
    long long *prefix;  // [batch + 1]: work items before each sequence
    int4 *seq;          // [batch]: AttSeq without hi
    float2 *scale;      // [ring]: (K scale, V scale without the probabilities' 2^14, so that the sums reach as far as
                        // fp32 does), K scale < 0: page not loaded
    uint64_t *full_k, *full_v, *empty_k, *empty_v;
    int *has_k, *has_v; // [ring]: number of the page whose turn the slot's K and V are at
    float *merge;       // [8 warps][8 NT rows][D + 4]
    float *ml;          // [8 warps][8 NT rows][2]
    int *ctrl;          // [0] abort
    uint8_t *ring;      // [ring][K page, V page]
};

__host__ __device__ constexpr int att_fixed_bytes(int D, int nt) {
    return ATT_WARPS * 8 * nt * (D + 4) * 4 + ATT_WARPS * 8 * nt * 2 * 4 + ATT_MAXRING * (8 + 32 + 8) + 16;
}
__host__ __device__ constexpr int att_seq_bytes(int batch) { return batch * 16 + (batch + 1) * 8; }

template <int D, int NT>
DEV AttShared att_shared(const AttParams &p) {
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
    at += 16;
    s.ml = reinterpret_cast<float *>(at);
    at += ATT_WARPS * 8 * NT * 2 * 4;
    s.merge = reinterpret_cast<float *>(at);
    at += ATT_WARPS * 8 * NT * (D + 4) * 4;
    s.seq = reinterpret_cast<int4 *>(at);
    s.prefix = reinterpret_cast<long long *>(s.seq + p.batch);
    const uint32_t used = (uint32_t)(at - mk_smem) + att_seq_bytes(p.batch);
    s.ring = mk_smem + ((used + 127) & ~127u);
    return s;
}

// Work item x belongs to the last sequence b with prefix[b] <= x that has any.
DEV int att_find(const long long *prefix, int batch, long long x) {
    int a = 0, z = batch;
    while (z - a > 1) {
        const int mid = (a + z) / 2;
        if (prefix[mid] <= x) a = mid;
        else z = mid;
    }
    return a;
}
// The pages of a sequence that the rows of one of its tiles see: [lo, hi).
template <int P, int RT>
DEV void att_tile_pages(const AttParams &p, const int4 &q, int tile, int &lo, int &hi) {
    const int rows = q.y * p.group;
    const int i0 = tile * RT / p.group, i1 = (min((tile + 1) * RT, rows) - 1) / p.group;
    const int top = q.z - q.y + i1, bottom = q.z - q.y + i0;
    hi = top < 0 ? 0 : top / P + 1;
    lo = att_least(bottom, p.window) / P;
}

// One range of pages of one unit, as every warp of the CTA walks them.  A page
// belongs to the CTA in whose range its first item lies.
struct AttSeg {
    int b, tile, h, pg, n;    // pages [pg, pg + n) of the sequence
    int q0, cnt, len;
    bool whole;               // the unit's every page
    bool head;                // the unit's first page among them
};

template <int P, int RT>
struct AttWalk {
    const AttParams &p;
    const AttShared &s;
    long long x, end;
    int b;
    DEV AttWalk(const AttParams &p_, const AttShared &s_) : p(p_), s(s_) {
        const long long total = s.prefix[p.batch];
        const int ctas = att_used<RT>(total, p.ctas);
        x = end = 0;
        if ((int)blockIdx.x < ctas) {
            x = att_div((long long)blockIdx.x * total, ctas);
            end = att_div((long long)(blockIdx.x + 1) * total, ctas);
        }
        b = att_find(s.prefix, p.batch, x);
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
            g.pg = q.w + first;
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
template <int D, int P, int RT>
DEV void att_produce(const AttParams &p, const AttShared &s) {
    constexpr int PAGE = P * D;
    const int lane = threadIdx.x % 32;
    uint8_t *dst = s.ring + (size_t)lane * 2 * PAGE;
    AttWalk<P, RT> walk(p, s);
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
                pg = g.pg + k;
                int lo, hi;
                att_tile_pages<P, RT>(p, make_int4(g.q0, g.cnt, g.len, 0), g.tile, lo, hi);
                if (pg >= lo && pg < hi) b = g.b;
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
DEV float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
DEV uint32_t half2_of(float lo, float hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
    return h;
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
DEV void att_consumer_bar() { asm volatile("bar.sync 1, %0;" ::"n"(ATT_WARPS * 32) : "memory"); }

template <int D, int P, int RT>
DEV void att_consume(const AttParams &p, const AttShared &s) {
    constexpr int NT = att_nt(RT), WT = RT / (8 * NT);  // 8-row tiles a warp, warps for a full tile
    constexpr int PAGE = P * D, RUN = P / 4, NM = P / 16, ND = D / 16, LD = D + 4;
    constexpr bool QS = NT > 1;  // the query operand in shared memory (registers would spill)
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g8 = lane / 4, t = lane % 4;
    AttWalk<P, RT> walk(p, s);
    AttSeg g;
    bool ok = true;
    int before = 0;  // pages of the CTA's ranges done
    while (walk.next(g)) {
        const int rows = g.cnt * p.group, base = g.len - g.cnt;
        // as many warps side by side as the tile's rows need (1, 2 or 4), the
        // others on other pages: group grp takes every ng-th page of the range
        const int side = att_side<RT>(rows - g.tile * RT);
        const int wt = warp % side, grp = warp / side, ng = ATT_WARPS / side;
        const int row0 = g.tile * RT + wt * 8 * NT;
        int st = (before + grp) % p.ring;  // ring slot and phase of this warp's next page
        uint32_t ph = ((before + grp) / p.ring) & 1;
        const auto settle = [&] {
            while (st >= p.ring) {
                st -= p.ring;
                ph ^= 1;
            }
        };
        const auto pos_of = [&](int r) { return r < rows ? base + r / p.group : -1; };  // a row sees [least, pos]
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
                all_hi = min(all_hi, base + tok);
                all_lo = max(all_lo, least_of(base + tok));
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
        if constexpr (QS) att_consumer_bar();
        for (int mine = before + grp; mine < before + g.n; mine += ng, st += ng, settle()) {
            const int pg = g.pg + mine - before;
            if (ok) ok = att_wait(p, s, &s.has_k[st], mine, &s.full_k[st], ph);
            ok = __all_sync(FULL, ok);
            if (!ok) continue;
            const float2 sc = s.scale[st];
            const bool there = sc.x >= 0.f || sc.x != sc.x;
            const uint8_t *kp = s.ring + (size_t)st * 2 * PAGE, *vp = kp + PAGE;
            if (there) {
                const bool edge = pg * P < all_lo || pg * P + P - 1 > all_hi;
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
                                    if (x > pos[n][e] || x < least) c[n][i][2 * u + e] = -INFINITY;
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
                                    see[k] = (x <= ps && x >= ls ? 0x3c00u : 0u) |
                                             (x + 1 <= ps && x + 1 >= ls ? 0x3c000000u : 0u);
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
            __syncwarp();
            if (ok && lane == 0) mbar_arrive_n(&s.empty_v[st], WT / side);
        }
        before += g.n;
        // merge the ng warps of each tile
        if constexpr (QS) att_consumer_bar();  // the query operand lies where the sums go
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
        att_consumer_bar();
        for (int i = threadIdx.x; i < RT * (D / 4); i += ATT_WARPS * 32) {
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
            if (g.whole) {
                const int64_t token = g.q0 + rr / p.group;
                const int hd = g.h * p.group + rr % p.group;
                const float inv = att_inverse(sum);
                *reinterpret_cast<uint2 *>(p.out + token * p.os_t + (int64_t)hd * p.os_h + 4 * d4) =
                    make_uint2(bf16_pair(acc.x * inv, acc.y * inv), bf16_pair(acc.z * inv, acc.w * inv));
                if (p.lse && d4 == 0)
                    p.lse[token * (p.group * p.c.hkv) + hd] = att_lse(big, sum);
            } else {
                const size_t slot = ((size_t)blockIdx.x * 2 + (g.head ? 1 : 0)) * RT + row;
                *reinterpret_cast<float4 *>(p.part_o + slot * D + 4 * d4) = acc;
                if (d4 == 0) *reinterpret_cast<float2 *>(p.part_ml + slot * 2) = make_float2(big, sum);
            }
        }
        att_consumer_bar();
    }
}

template <int D, int P, int RT>
__global__ void __launch_bounds__(ATT_THREADS, 1) cache_attend_kernel(const AttParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    const AttShared s = att_shared<D, att_nt(RT)>(p);
    const int tid = threadIdx.x;
    for (int b = tid; b < p.batch; b += ATT_THREADS) {
        const AttSeq q = att_seq<P>(p, b, blockIdx.x == 0);
        s.prefix[b + 1] = att_items<RT>(p, q.cnt, q.hi - q.lo);
        s.seq[b] = make_int4(q.q0, q.cnt, q.len, q.lo);
    }
    if (tid >= ATT_THREADS - 32 && tid - (ATT_THREADS - 32) < p.ring) {
        const int i = tid - (ATT_THREADS - 32);
        s.has_k[i] = s.has_v[i] = -1;
        mbar_init(&s.full_k[i], 2);
        mbar_init(&s.full_v[i], 1);
        mbar_init(&s.empty_k[i], RT / (8 * att_nt(RT)));
        mbar_init(&s.empty_v[i], RT / (8 * att_nt(RT)));
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 0) s.ctrl[0] = 0;
    att_running(s.prefix, p.batch);
    if (tid >= ATT_WARPS * 32) att_produce<D, P, RT>(p, s);
    else att_consume<D, P, RT>(p, s);
}

// One warp per query row: rows that see nothing get zeros, rows whose pages
// two or more CTAs shared are merged, in the order of the CTAs; the others
// are written already.  All that does not need the main kernel's results (the
// sequences' running page counts again, the row's sequence) runs while that
// one still does.
template <int D, int P, int RT>
__global__ void __launch_bounds__(256) cache_attend_merge(const AttParams p) {
    long long *prefix = reinterpret_cast<long long *>(mk_smem);
    const int tid = threadIdx.x, lane = tid % 32, heads = p.group * p.c.hkv;
    for (int b = tid; b < p.batch; b += 256) {
        const AttSeq q = att_seq<P>(p, b, false);
        prefix[b + 1] = att_items<RT>(p, q.cnt, q.hi - q.lo);
    }
    att_running(prefix, p.batch);
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
    const AttSeq s = att_seq<P>(p, b, false);
    const int np = s.hi - s.lo, h = head / p.group, r = (token - s.q0) * p.group + head % p.group;
    bool todo = w < (int64_t)p.tokens * heads && token >= s.q0 && token < s.q0 + s.cnt;
    int c0 = 0, c1 = -1;
    if (todo && np > 0) {
        const int rows = s.cnt * p.group, tile = r / RT, side = att_side<RT>(rows - tile * RT);
        const long long total = prefix[p.batch];
        constexpr int FIXED = att_fixed_items(RT);
        const long long x0 = prefix[b] + (long long)tile * p.c.hkv * (np * att_side<RT>(RT) + FIXED) +
                             h * ((long long)np * side + FIXED) + FIXED;  // the first page's item
        const int ctas = att_used<RT>(total, p.ctas);
        c0 = att_owner(x0, total, ctas);
        c1 = att_owner(x0 + (long long)(np - 1) * side, total, ctas);
        todo = c0 != c1;
    }
    // every thread waits: this grid must not be done before the main kernel is
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!todo) return;
    const auto slot = [&](int c) { return ((size_t)c * 2 + (c == c0 ? 1 : 0)) * RT + r % RT; };  // c0 has the unit's head
    constexpr int V = D / 32;
    float acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    float big = -INFINITY, sum = 0.f;
    for (int c = c0; c <= c1; c += 32) {  // the maxima first, 32 CTAs at a time
        const int mine = c + lane;
        const float2 ml = mine <= c1 ? *reinterpret_cast<const float2 *>(p.part_ml + slot(mine) * 2)
                                     : make_float2(-INFINITY, 0.f);
        const float top = fmaxf(big, warp_max(ml.x)), mu = top == -INFINITY ? 0.f : top;
        const float a = exp2_fast(big - mu), e = exp2_fast(ml.x - mu);
        big = top;
        sum *= a;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] *= a;
        const int n = min(32, c1 - c + 1);
#pragma unroll 4
        for (int j = 0; j < n; ++j) {
            const float ej = __shfl_sync(FULL, e, j), lj = __shfl_sync(FULL, ml.y, j);
            const float *o = p.part_o + slot(c + j) * D + lane * V;
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

struct AttPlan {
    int rt, ctas;
    uint64_t ml_bytes, o_bytes;
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
    // no more CTAs than pages there can be (all tiles' together, each as many items as it has warps side by side)
    const int64_t side = pl.rt == 64 ? 4 : pl.rt == 32 ? 2 : 1;
    const int64_t tiles = a->batch + (int64_t)a->tokens * (a->q_heads / c->kv_heads) / pl.rt;
    pl.ctas = (int)std::min<int64_t>(sms, std::max<int64_t>(1, std::min<int64_t>(tiles * c->kv_heads, INT32_MAX) * (a->table_width * side + att_fixed_items(pl.rt))));
    pl.ml_bytes = ((uint64_t)pl.ctas * 2 * pl.rt * 8 + 255) / 256 * 256;
    pl.o_bytes = (uint64_t)pl.ctas * 2 * pl.rt * c->head_dim * 4;
    return MK_OK;
}

using AttFn = void (*)(const AttParams);
template <int D, int P>
static AttFn att_kernel(int rt) {
    return rt == 8 ? cache_attend_kernel<D, P, 8> : rt == 16 ? cache_attend_kernel<D, P, 16>
         : rt == 32 ? cache_attend_kernel<D, P, 32> : cache_attend_kernel<D, P, 64>;
}
template <int D, int P>
static AttFn att_merge_kernel(int rt) {
    return rt == 8 ? cache_attend_merge<D, P, 8> : rt == 16 ? cache_attend_merge<D, P, 16>
         : rt == 32 ? cache_attend_merge<D, P, 32> : cache_attend_merge<D, P, 64>;
}

}  // namespace mk

using namespace mk;

extern "C" {

int mk_cache_attend_workspace(const mk_cache_desc *cache, const mk_attend_desc *attend, uint64_t *bytes) {
    AttPlan pl;
    if (!bytes) return set_error(MK_ERR_INVALID, "bytes is null");
    if (int rc = att_plan(cache, attend, pl)) return rc;
    *bytes = pl.ml_bytes + pl.o_bytes;
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
    if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < pl.ml_bytes + pl.o_bytes)
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
    p.part_ml = reinterpret_cast<float *>(ws);
    p.part_o = reinterpret_cast<float *>(ws + pl.ml_bytes);
    const int fixed = att_fixed_bytes(D, att_nt(pl.rt)) + att_seq_bytes(p.batch) + 128;
    p.ring = std::min(ATT_MAXRING, (SERVE_SMEM - fixed) / (2 * P * D));
    const int smem = fixed + p.ring * 2 * P * D;
    AttFn f = D == 64 ? (P == 32 ? att_kernel<64, 32>(pl.rt) : att_kernel<64, 64>(pl.rt))
                      : (P == 32 ? att_kernel<128, 32>(pl.rt) : att_kernel<128, 64>(pl.rt));
    static std::atomic<uint32_t> ready[SERVE_MAX_DEVICES];
    const int variant = (D == 128 ? 8 : 0) + (P == 64 ? 4 : 0) + (pl.rt == 8 ? 0 : pl.rt == 16 ? 1 : pl.rt == 32 ? 2 : 3);
    if (int rc = serve_prepare(reinterpret_cast<const void *>(f), ready, variant, false)) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    f<<<pl.ctas, ATT_THREADS, smem, st>>>(p);
    cudaError_t e = cudaGetLastError();
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
    cfg.dynamicSmemBytes = (size_t)(p.batch + 1) * 8;
    AttFn mf = D == 64 ? (P == 32 ? att_merge_kernel<64, 32>(pl.rt) : att_merge_kernel<64, 64>(pl.rt))
                       : (P == 32 ? att_merge_kernel<128, 32>(pl.rt) : att_merge_kernel<128, 64>(pl.rt));
    e = cudaLaunchKernelEx(&cfg, mf, (const AttParams)p);
    return e == cudaSuccess ? MK_OK : serve_cuda_fail(e, "attention merge launch");
}

}  // extern "C"
