// Attention of a group's rows over the pages that its sequences share: the
// first of cache attention's launches where groups are large (attend.cu then
// does the sequences' own pages and joins both).
//
// Mathematics.  As in attend.cu: one pass over the pages with the running
// maximum m and sum l of the softmax in log2 units, sums in fp32, scores K q,
// outputs P V.  Every row sees every token, so there are no masks.
//
// Matrix products.  tcgen05.mma kind::f16 on tiles of 128 rows (the group's
// tokens x q heads of one kv head): S = Q K^T with Q in tensor memory and a
// page's K in shared memory, then O += P V with P in tensor memory.  Codes are
// expanded to f16 (exact) by eight warps on their way from the ring the pages
// land in to the swizzled tiles the products read; a row of Q is scaled by a
// power of two into f16's range.
//
// One reference.  P and O are relative to a row's reference r, which is the
// first page's largest s + log2(the page's V scale) and follows a larger one only
// when that is 2^8 above it: then O is rescaled in tensor memory, and else nothing
// is.  P = 2^(s + log2 vs - r + 7) holds the V scale, so that pages of different
// scales add up in one accumulator; it stays below 2^15, and what it rounds away
// is 2^-11 of itself or 2^-32 of the reference.  The sum is relative to the
// largest s and takes the page's P as they are in fp32, without the scale.
//
// Fewer rows.  The tile's 128 lanes hold two copies of up to 64 rows, or four of
// up to 32: each copy takes the softmax of its share of a page's tokens, the
// others' columns of its P staying zero, and the copies are joined at the end.
// The products cost the same, and the softmax, one lane a row, a half or quarter.
//
// Roles.  Two streams of four softmax warps take pages in turn, so that one's
// products run during the other's softmax; four warps each expand K and V; one
// producer (bulk copies); one warp issues the products.
//
// What bounds it: 0.9 us a page of 64 tokens and 128 dims and tile of 128 rows,
// 4.7 TFLOP/s an SM.  The products alone are 512 clocks (measured: 64 for 128 x
// 128 x 16); the rest is shared memory (a page's codes land, are read, and are
// written twice as large, and the products read them: some 770 wavefronts of 128
// bytes without conflicts) and the way of a page through scores, softmax and
// outputs, of which tensor memory holds two.  Tried and slower: a third pair of tiles, all 64
// scores in registers, V expanded by integer instructions, spinning waits.
//
// Work split.  As in attend.cu: the pages of all (group, tile, kv head) are one
// axis cut into equal ranges, one per CTA; what a CTA boundary cuts is merged
// by the call's last launch, in the order of the CTAs.
#include "dev_attend.cuh"

namespace mk {

constexpr int PRE_THREADS = 640;
constexpr int PRE_ISSUER = 17;  // warp
constexpr int PRE_MAXRING = 32;

// Tensor memory columns, P tokens a page: O of both streams, S, P, then Q.
constexpr int PRE_O = 0, PRE_S = 256, PRE_P = 384, PRE_Q = 448;

struct PreShared {
    long long *prefix;  // [ngroups + 1]: work items before each group
    int4 *unit;         // [ngroups]: first query row, query tokens, pages, leading sequence
    AttGroups groups;
    float2 *in_scale;   // [ring]: K scale (below 0: page not loaded), log2 of the V scale
    float2 *scale;      // [4]: of the page on its way through the products, by page number % 4
    float *qf;          // [128]: a row's factor
    float *ml;          // [256][2]
    float *merge;       // [256][36]; before that, the queries' rows
    float **to;         // [128]: where a row's outputs go
    uint64_t *full, *empty;                                     // [ring]
    // [2], by stream: K's tile is written and the scores before are read; S is
    // there; V's tile and P are written; O is there.  A tile is free again when
    // its product is.
    uint64_t *s_ready, *s_done, *o_ready, *o_done;
    uint64_t *q_full, *q_empty, *drain;
    int *ctrl;          // [0] abort, [1] tensor memory address, [2] CTAs that share the work
    unsigned long long *total;  // items of the launch beside this one
    uint8_t *tiles;     // [2][K f16, V f16]
    uint8_t *ring;      // [ring][K page, V page]
};

__host__ __device__ constexpr int pre_fixed_bytes(int ngroups) {
    return (ngroups + 1) * 8 + ngroups * 16 + att_group_bytes(ngroups) + PRE_MAXRING * 8 + 4 * 8 + 128 * 4 + 128 * 8 + 256 * 8 +
           256 * 36 * 4 + (2 * PRE_MAXRING + 4 * 2 + 3) * 8 + 24 + 64;
}

template <int D, int P>
DEV PreShared pre_shared(const AttParams &p) {
    PreShared s;
    uint8_t *at = mk_smem;
    const auto take = [&](size_t bytes) {
        uint8_t *x = at;
        at += bytes;
        return x;
    };
    s.tiles = take(4 * P * D * 2);  // at 1024-byte boundaries: the dynamic shared memory starts at one (checked)
    s.ring = take((size_t)p.ring * 2 * P * D);
    s.merge = reinterpret_cast<float *>(take(256 * 36 * 4));
    s.ml = reinterpret_cast<float *>(take(256 * 8));
    s.qf = reinterpret_cast<float *>(take(128 * 4));
    s.to = reinterpret_cast<float **>(take(128 * 8));
    s.unit = reinterpret_cast<int4 *>(take(p.ngroups * 16));
    s.in_scale = reinterpret_cast<float2 *>(take(PRE_MAXRING * 8));
    s.scale = reinterpret_cast<float2 *>(take(4 * 8));
    s.full = reinterpret_cast<uint64_t *>(take((2 * PRE_MAXRING + 4 * 2 + 3) * 8));
    s.empty = s.full + PRE_MAXRING;
    s.s_ready = s.empty + PRE_MAXRING;
    s.s_done = s.s_ready + 2;
    s.o_ready = s.s_done + 2;
    s.o_done = s.o_ready + 2;
    s.q_full = s.o_done + 2;
    s.q_empty = s.q_full + 1;
    s.drain = s.q_empty + 1;
    s.prefix = reinterpret_cast<long long *>(take((p.ngroups + 1) * 8));
    s.total = reinterpret_cast<unsigned long long *>(take(8));
    s.ctrl = reinterpret_cast<int *>(take(16));
    s.groups = att_groups_at(at, p.ngroups);
    return s;
}

// ---- tensor memory and products
// True in one thread of a whole warp, always the same.
DEV bool pre_elect() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(e));
    return e != 0;
}
DEV void pre_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
DEV void pre_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(saddr(bar)) : "memory");
}
DEV void pre_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
DEV void pre_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
DEV void pre_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
DEV void pre_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// f16 A and B (both K-major), fp32 D, 128 x n
__host__ __device__ constexpr uint32_t pre_idesc(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(PRE_ROWS >> 4) << 24); }
// K-major operand of rows of 128 (64) bytes, swizzled by as much: 8-row groups 1024 (512) bytes apart.
template <bool WIDE>
DEV uint64_t pre_desc(uint32_t addr) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)((WIDE ? 1024 : 512) >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)(WIDE ? 2 : 4) << 61;
}
// A warp's 32 lanes x N columns.
template <int N>
DEV void pre_ld(uint32_t addr, uint32_t (&r)[N]) {
    static_assert(N == 8 || N == 16 || N == 32, "");
    if constexpr (N == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(addr));
    else if constexpr (N == 16)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
            : "r"(addr));
    else
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
            "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
            : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
              "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]),
              "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]),
              "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
            : "r"(addr));
}
template <int N>
DEV void pre_st(uint32_t addr, const uint32_t (&r)[N]) {
    static_assert(N == 4 || N == 8 || N == 16, "");
    if constexpr (N == 4)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]) : "memory");
    else if constexpr (N == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
                     "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    else
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(addr),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
            "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
            : "memory");
}

// ---- waits
// Bounded (about two seconds); false: it ran out here or elsewhere in the CTA.
DEV bool pre_wait(const AttParams &p, const PreShared &s, uint64_t *bar, uint32_t parity) {
    if (mbar_test(bar, parity)) return true;
    for (int i = 0; i < 20000; ++i) {
        if (mbar_wait_hint(bar, parity, 100000)) return true;
        if (*reinterpret_cast<volatile int *>(s.ctrl)) return false;
    }
    note_failure(p.c.status, MK_ERR_TIMEOUT, -1, blockIdx.x, -1);
    *reinterpret_cast<volatile int *>(s.ctrl) = 1;
    return false;
}
// By a whole warp: the same answer in all lanes.
DEV bool pre_wait_warp(const AttParams &p, const PreShared &s, uint64_t *bar, uint32_t parity) {
    return __all_sync(FULL, pre_wait(p, s, bar, parity));
}

// ---- the CTA's range, as every role walks it
struct PreSeg {
    int g, tile, h, pg, n;  // pages [pg, pg + n) of a unit
    int q0, rows, lead;     // the group's first query token, its rows of one kv head, whose table row
    bool whole, head;       // all of the unit's pages; its first among them
    DEV int tile_rows() const { return min(PRE_ROWS, rows - tile * PRE_ROWS); }
    DEV int copies() const { const int n = tile_rows(); return n <= 32 ? 4 : n <= 64 ? 2 : 1; }
};
struct PreWalk {
    const AttParams &p;
    const PreShared &s;
    long long x = 0, end = 0;
    int g;
    DEV PreWalk(const AttParams &p_, const PreShared &s_) : p(p_), s(s_) {
        const long long total = s.prefix[p.ngroups];
        const int ctas = pre_used(total, s.ctrl[2]);
        if ((int)blockIdx.x < ctas) {
            x = att_div((long long)blockIdx.x * total, ctas);
            end = att_div((long long)(blockIdx.x + 1) * total, ctas);
        }
        g = att_find(s.prefix, p.ngroups, x);
    }
    DEV bool next(PreSeg &o) {
        while (x < end) {
            while (s.prefix[g + 1] <= x) ++g;
            const int4 u = s.unit[g];
            const int np = u.z, items = np + PRE_FIXED;
            const long long r = x - s.prefix[g];
            const int unit = (int)att_div(r, items), within = (int)(r - (long long)unit * items);
            const long long left = items - within;  // items to the unit's end
            const int first = max(0, within - PRE_FIXED);
            const int until = left <= end - x ? np : max(0, within + (int)(end - x) - PRE_FIXED);
            x += min(left, end - x);
            if (first >= until) continue;
            o.g = g;
            o.tile = unit / p.c.hkv;
            o.h = unit - o.tile * p.c.hkv;
            o.pg = first;
            o.n = until - first;
            o.q0 = u.x;
            o.rows = u.y * p.group;
            o.lead = u.w;
            o.whole = o.n == np;
            o.head = first == 0;
            return true;
        }
        return false;
    }
};

// ---- producer warp: lane i looks up the i-th of 32 pages, then each issues its own in turn
template <int D, int P>
DEV void pre_produce(const AttParams &p, const PreShared &s) {
    constexpr int PAGE = P * D;
    const int lane = threadIdx.x % 32;
    PreWalk walk(p, s);
    PreSeg g;
    bool more = walk.next(g), ok = true;
    int before = 0, slot = 0;
    uint32_t round = 0;
    for (int base = 0; more && ok; base += 32) {
        int id = -1, h = 0;
        bool want = false;
        while (more) {
            const int k = base + lane - before;
            if (k >= 0 && k < g.n) {
                want = true;
                h = g.h;
                id = p.table[(size_t)g.lead * p.width + g.pg + k];
                if ((unsigned)id >= (unsigned)p.c.pages) {
                    note_failure(p.c.status, MK_ERR_DEVICE_CHECK, g.lead, (g.pg + k) * P, id);
                    id = -1;
                }
            }
            if (before + g.n > base + 32) break;
            before += g.n;
            more = walk.next(g);
        }
        const size_t at = (size_t)(id < 0 ? 0 : id) * p.c.hkv + h;
        float2 sc = make_float2(-1.f, 0.f);
        if (id >= 0) {
            // a power of two, or 0 for a page of zeros (any scale does then), or NaN
            const float v = p.c.vs[at];
            sc = make_float2(p.c.ks[at], v == 0.f ? -120.f : v != v ? v : (float)((int)(__float_as_uint(v) >> 23 & 255) - 127));
        }
        const int n = __popc(__ballot_sync(FULL, want));
        for (int i = 0; i < n && ok; ++i) {
            if (lane == i) {
                ok = round == 0 || pre_wait(p, s, &s.empty[slot], (round & 1) ^ 1);
                if (ok) {
                    s.in_scale[slot] = sc;
                    uint8_t *dst = s.ring + (size_t)slot * 2 * PAGE;
                    if (id >= 0) {
                        mbar_expect_tx(&s.full[slot], 2 * PAGE);
                        bulk_g2s_plain(dst, p.c.k + at * PAGE, PAGE, &s.full[slot]);
                        bulk_g2s_plain(dst + PAGE, p.c.v + at * PAGE, PAGE, &s.full[slot]);
                    } else {
                        mbar_arrive(&s.full[slot]);
                    }
                }
            }
            ok = __shfl_sync(FULL, ok, i);
            if (ok && ++slot == p.ring) {
                slot = 0;
                ++round;
            }
        }
    }
    // the copies in flight land before the CTA ends, also where the warps that wanted them have given up
    if (lane < p.ring) {
        const uint32_t fills = round + (lane < slot ? 1 : 0);
        for (int i = 0; i < 200 && fills && !mbar_wait_hint(&s.full[lane], (fills - 1) & 1, 1000000); ++i) {
        }
    }
}

// ---- converting warps: a landed page's codes as f16 into the products' tiles
// 16 codes as two 16-byte pieces
DEV void pre_expand(uint4 x, uint4 &lo, uint4 &hi) {
    e4m3x4_to_half2(x.x, lo.x, lo.y);
    e4m3x4_to_half2(x.y, lo.z, lo.w);
    e4m3x4_to_half2(x.z, hi.x, hi.y);
    e4m3x4_to_half2(x.w, hi.z, hi.w);
}
template <int D, int P, bool VALUES>
DEV void pre_convert(const AttParams &p, const PreShared &s) {
    constexpr int PAGE = P * D, N = PAGE / 16 / 128;  // 16-byte pieces of codes per thread
    const int tid = threadIdx.x % 128, lane = tid % 32;
    PreWalk walk(p, s);
    PreSeg g;
    int total = 0;
    while (walk.next(g)) total += g.n;
    uint64_t *ready = VALUES ? s.o_ready : s.s_ready, *done = VALUES ? s.o_done : s.s_done;
    int slot = 0;
    uint32_t round = 0;
    for (int n = 0; n < total; ++n) {
        const int x = n & 1;
        if (!pre_wait_warp(p, s, &s.full[slot], round & 1)) return;
        const float2 sc = s.in_scale[slot];
        const bool there = sc.x >= 0.f || sc.x != sc.x;
        const uint8_t *raw = s.ring + (size_t)slot * 2 * PAGE + (VALUES ? PAGE : 0);
        uint8_t *tile = s.tiles + (size_t)x * 4 * PAGE + (VALUES ? 2 * PAGE : 0);
        uint4 in[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
            in[i] = there ? *reinterpret_cast<const uint4 *>(raw + (i * 128 + tid) * 16) : make_uint4(0, 0, 0, 0);
        if (n > 1 && !pre_wait_warp(p, s, &done[x], ((n >> 1) & 1) ^ 1)) return;  // the tile's last product
        if (!VALUES && tid == 0) s.scale[n & 3] = sc;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int at = i * 128 + tid;
            uint4 lo, hi;
            pre_expand(in[i], lo, hi);
            if constexpr (VALUES) {  // dim d, tokens 16 j ..
                const int d = at / (P / 16), j = at % (P / 16), sw = P == 64 ? d & 7 : (d >> 1) & 3;
                uint8_t *row = tile + d * (P * 2);
                *reinterpret_cast<uint4 *>(row + (((2 * j) ^ sw) << 4)) = lo;
                *reinterpret_cast<uint4 *>(row + (((2 * j + 1) ^ sw) << 4)) = hi;
            } else {  // token t, dims 16 j ..: block j / 4, pieces 2 (j % 4) and the next of its 128-byte row
                const int t = at / (D / 16), j = at % (D / 16), c = 2 * (j & 3);
                uint8_t *row = tile + (j >> 2) * (P * 128) + t * 128;
                // blocks lie a multiple of 1024 bytes apart: the second one's lanes store their second piece first
                const int other = j >> 2;
                *reinterpret_cast<uint4 *>(row + (((c + other) ^ (t & 7)) << 4)) = other ? hi : lo;
                *reinterpret_cast<uint4 *>(row + (((c + 1 - other) ^ (t & 7)) << 4)) = other ? lo : hi;
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&ready[x]);
            mbar_arrive(&s.empty[slot]);
        }
        if (++slot == p.ring) {
            slot = 0;
            ++round;
        }
    }
}

// ---- the products, issued by one elected thread of a warp
template <int D, int P>
DEV void pre_products(const AttParams &p, const PreShared &s, uint32_t tmem) {
    constexpr int PAGE = P * D;
    if (!pre_elect()) return;
    const uint64_t k_tile = pre_desc<true>(saddr(s.tiles)), v_tile = pre_desc<P == 64>(saddr(s.tiles) + 2 * PAGE);
    PreWalk walk(p, s);
    PreSeg g;
    int n = 0;  // pages done
    uint32_t seg = 0;
    bool ok = true;
    const auto scores = [&](int k) {
        const int x = k & 1;
        ok = ok && pre_wait(p, s, &s.s_ready[x], (k >> 1) & 1);
        if (!ok) return;
        pre_fence_after();
#pragma unroll
        for (int i = 0; i < D / 16; ++i)  // (descriptors count 16 bytes)
            pre_mma(tmem + PRE_S + x * 64, tmem + PRE_Q + i * 8, k_tile + (x * 4 * PAGE + (i / 4) * (P * 128) + (i % 4) * 32) / 16,
                    pre_idesc(P), i > 0);
        pre_commit(&s.s_done[x]);
    };
    const auto outputs = [&](int k, bool first) {
        const int x = k & 1;
        ok = ok && pre_wait(p, s, &s.o_ready[x], (k >> 1) & 1);
        if (!ok) return;
        pre_fence_after();
#pragma unroll
        for (int i = 0; i < P / 16; ++i)
            pre_mma(tmem + PRE_O + x * 128, tmem + PRE_P + x * 32 + i * 8, v_tile + (x * 4 * PAGE + i * 32) / 16, pre_idesc(D),
                    i > 0 || !first);
        pre_commit(&s.o_done[x]);
    };
    for (; ok && walk.next(g); ++seg) {
        ok = pre_wait(p, s, s.q_full, seg & 1);
        // scores two pages ahead: a stream's next ones are there when its softmax is done
        for (int i = 0; i < g.n + 2 && ok; ++i) {
            if (i < g.n) scores(n + i);
            if (i + 1 == g.n && ok) pre_commit(s.q_empty);
            if (i > 1) outputs(n + i - 2, i < 4);
        }
        n += g.n;
    }
    // what was issued ends before tensor memory is freed
    pre_commit(s.drain);
    for (int i = 0; i < 200 && !mbar_wait_hint(s.drain, 0, 1000000); ++i) {
    }
}

// ---- softmax warps
// A row's state: the reference of P and O (of s + log2 of V scales), the largest
// s, and the sum of 2^s relative to that.
struct PreRow {
    float ref, top, sum;
};
// One page's scores to probabilities: this thread's row, CN tokens.  `taken` is
// called when the scores are read, `settle` before P is written, with what O has
// to be multiplied by (1: nothing).
template <int CN, typename Taken, typename Settle>
DEV void pre_softmax(uint32_t s_addr, uint32_t p_addr, float fk, float lv, PreRow &w, const Taken &taken, const Settle &settle) {
    constexpr int W = CN < 32 ? CN : 32;  // scores in registers at a time
    uint32_t r[W];
    float mx = -INFINITY;
#pragma unroll
    for (int c = 0; c < CN; c += W) {
        pre_ld(s_addr + c, r);
        pre_wait_ld();
#pragma unroll
        for (int i = 0; i < W; ++i) mx = fmaxf(mx, __uint_as_float(r[i]));
    }
    mx *= fk;
    const float top = fmaxf(w.top, mx), mu = top == -INFINITY ? 0.f : top;
    w.sum *= exp2_fast(w.top - mu);
    w.top = top;
    const float to = mx + (lv == lv ? lv : 0.f);
    float back = 1.f;
    if (!(to <= w.ref + 8.f)) {  // (the first page; a NaN score leaves the reference)
        back = to > w.ref ? exp2_fast(w.ref - to) : 1.f;
        w.ref = to > w.ref ? to : w.ref;
    }
    const float at = w.ref == -INFINITY ? 0.f : w.ref, off = lv + 7.f - at;
    // scales so far apart that P may be 0 where the sum is not (or a NaN scale,
    // which makes outputs NaN, not the sum): the sum's terms by themselves
    const bool apart = !(to >= at - 60.f) || lv != lv, some = __any_sync(FULL, apart);
    if (CN == W && !some) taken();
    float sum = 0.f;
#pragma unroll
    for (int c = CN - W; c >= 0; c -= W) {  // the last part is in registers
        if (c < CN - W) {
            pre_ld(s_addr + c, r);
            pre_wait_ld();
            if (c == 0 && !some) taken();
        }
        uint32_t h[W / 2];
#pragma unroll
        for (int i = 0; i < W; i += 2) {
            const float a = exp2_fast(fmaf(__uint_as_float(r[i]), fk, off)), b = exp2_fast(fmaf(__uint_as_float(r[i + 1]), fk, off));
            sum += a + b;
            h[i / 2] = half2_of(a, b);
        }
        if (c == CN - W) settle(back);
        pre_st(p_addr + c / 2, h);
    }
    const float here = sum * exp2_fast(-off - mu);
    float alone = 0.f;
    if (some) {
#pragma unroll 1
        for (int c = 0; c < CN; c += 8) {
            uint32_t t[8];
            pre_ld(s_addr + c, t);
            pre_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) alone += exp2_fast(fmaf(__uint_as_float(t[i]), fk, -mu));
        }
        taken();
    }
    w.sum += apart ? alone : here;
}

DEV void pre_bar() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <int D, int P>
DEV void pre_rows(const AttParams &p, const PreShared &s, uint32_t tmem) {
    const int x = threadIdx.x / 128, tid = threadIdx.x % 128, lane = tid % 32, warp = tid / 32;
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    const uint32_t s_addr = lanes + PRE_S + x * 64, p_addr = lanes + PRE_P + x * 32, o_addr = lanes + PRE_O + x * 128;
    PreWalk walk(p, s);
    PreSeg g;
    int n = 0;  // pages before the segment
    uint32_t seg = 0;
    bool ok = true;  // a warp that gives up still takes its place at the barriers
    if (lane == 0) mbar_arrive(&s.s_ready[x]);  // no scores before the first
    for (; walk.next(g); ++seg, n += g.n) {
        const int copies = g.copies(), each = PRE_ROWS / copies, copy = tid / each, rows = g.tile_rows();
        if (x == 0) {  // the segment's queries: row by row to shared memory, then a row per lane
            constexpr int LINE = D * 2 + 16;
            uint8_t *stage = reinterpret_cast<uint8_t *>(s.merge) + warp * 32 * LINE;
            const int row0 = g.tile * PRE_ROWS + (warp * 32) % each, there = rows - (warp * 32) % each;
            constexpr int LANES = D / 8, AT_ONCE = 32 / LANES;  // lanes to a row of 16-byte pieces
            constexpr int BATCH = 32 / AT_ONCE;  // all at once: one round trip
#pragma unroll
            for (int i = 0; i < 32; i += AT_ONCE * BATCH) {
                uint4 q[BATCH];
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {  // (rows behind the last: it again, then zeros)
                    const int r = row0 + max(0, min(i + k * AT_ONCE + lane / LANES, there - 1)), tok = r / p.group;
                    q[k] = make_uint4(0, 0, 0, 0);
                    const int64_t at = (int64_t)(g.q0 + tok) * p.qs_t + (int64_t)(g.h * p.group + r - tok * p.group) * p.qs_h;
                    if (there > 0) q[k] = __ldg(reinterpret_cast<const uint4 *>(p.q + at) + lane % LANES);
                }
#pragma unroll
                for (int k = 0; k < BATCH; ++k) {
                    const int mine = i + k * AT_ONCE + lane / LANES;
                    *reinterpret_cast<uint4 *>(stage + mine * LINE + lane % LANES * 16) = mine < there ? q[k] : make_uint4(0, 0, 0, 0);
                }
            }
            __syncwarp();
            const uint4 *row = reinterpret_cast<const uint4 *>(stage + lane * LINE);
            uint32_t big = 0;
            const auto most = [&](uint32_t w) { big = max(big, max((w << 16) & 0x7fffffffu, w & 0x7fff0000u)); };
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
                const uint4 q = row[i];
                most(q.x), most(q.y), most(q.z), most(q.w);
            }
            // times 2^(14 - exponent): the row's largest value lands in [2^14, 2^15)
            const int up = min(max(268 - (int)(big >> 23), 1), 253);
            const float sc = __uint_as_float((uint32_t)up << 23);
            const auto pair = [&](uint32_t w) { return half2_of(__uint_as_float(w << 16) * sc, __uint_as_float(w & 0xffff0000u) * sc); };
            if (seg > 0 && ok) ok = pre_wait_warp(p, s, s.q_empty, (seg - 1) & 1);
            pre_fence_after();
#pragma unroll
            for (int c = 0; c < D / 2; c += 16) {
                uint32_t h[16];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 q = row[c / 4 + i];
                    h[4 * i] = pair(q.x), h[4 * i + 1] = pair(q.y), h[4 * i + 2] = pair(q.z), h[4 * i + 3] = pair(q.w);
                }
                pre_st(lanes + PRE_Q + c, h);
            }
            s.qf[tid] = big >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : __uint_as_float((uint32_t)(254 - up) << 23);
            pre_wait_st();
            pre_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(s.q_full);
        }
        if (copies > 1) {  // the other copies' columns stay zero
            const uint32_t zero[16] = {};
#pragma unroll
            for (int c = 0; c < P / 2; c += 16) pre_st(p_addr + c, zero);
            pre_wait_st();
        }
        if (ok) ok = pre_wait_warp(p, s, s.q_full, seg & 1);
        const float qf = s.qf[tid] * p.scale_log2;
        PreRow w{-INFINITY, -INFINITY, 0.f};
        int last = -1;  // the stream's page before
        const auto taken = [&] {  // the scores' columns may be written again
            pre_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.s_ready[x]);
        };
        // P's and O's earlier product is done; O relative to a new reference
        const auto settle = [&](float back) {
            if (last < 0) return;
            ok = pre_wait_warp(p, s, &s.o_done[x], (last >> 1) & 1);
            if (!ok || __all_sync(FULL, back == 1.f)) return;
            pre_fence_after();
#pragma unroll
            for (int c = 0; c < D; c += 16) {
                uint32_t r[16];
                pre_ld(o_addr + c, r);
                pre_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * back);
                pre_st(o_addr + c, r);
            }
        };
        for (int k = n + ((n ^ x) & 1); k < n + g.n && ok; k += 2) {
            ok = pre_wait_warp(p, s, &s.s_done[x], (k >> 1) & 1);
            if (!ok) break;
            pre_fence_after();
            const float2 sc = s.scale[k & 3];
            if (sc.x >= 0.f || sc.x != sc.x) {
                const float fk = qf * sc.x;
                if (copies == 1) pre_softmax<P>(s_addr, p_addr, fk, sc.y, w, taken, settle);
                else if (copies == 2) pre_softmax<P / 2>(s_addr + copy * (P / 2), p_addr + copy * (P / 4), fk, sc.y, w, taken, settle);
                else pre_softmax<P / 4>(s_addr + copy * (P / 4), p_addr + copy * (P / 8), fk, sc.y, w, taken, settle);
            } else {  // a page that is not loaded: as if its tokens were masked
                taken();
                settle(1.f);
                const uint32_t zero[16] = {};
#pragma unroll
                for (int c = 0; c < P / 2; c += 16) pre_st(p_addr + c, zero);
            }
            pre_wait_st();
            pre_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.o_ready[x]);
            last = k;
        }
        if (last >= 0 && ok) ok = pre_wait_warp(p, s, &s.o_done[x], (last >> 1) & 1);
        pre_fence_after();
        const float m = w.top, l = w.sum * 0x1p14f;  // as attend.cu has them: the sum of 2^(s - m + 14), outputs relative to m

        // join the copies of both streams, 32 dims at a time
        constexpr int LD = 36;
        *reinterpret_cast<float2 *>(s.ml + threadIdx.x * 2) = make_float2(m, l);
        pre_bar();
        const int parts = 2 * copies;  // row r of the tile: threads r + i * each
        float big = -INFINITY;
        for (int i = 0; i < parts; ++i) big = fmaxf(big, s.ml[(tid % each + i * each) * 2]);
        // O times 2^(ref - 7 - big), in two steps (a V scale may be 2^120)
        const float part = exp2_fast(0.5f * (w.ref - 7.f - (big == -INFINITY ? 0.f : big)));
        if (threadIdx.x < rows) {  // (rows <= each: this thread's row is threadIdx.x)
            float sum = 0.f;
            for (int i = 0; i < parts; ++i) {
                const float2 y = *reinterpret_cast<const float2 *>(s.ml + (threadIdx.x + i * each) * 2);
                sum = fmaf(y.y, exp2_fast(y.x - (big == -INFINITY ? 0.f : big)), sum);
            }
            const int rr = g.tile * PRE_ROWS + threadIdx.x, tok = rr / p.group;
            const size_t to = g.whole ? (((size_t)p.tokens + g.q0 + tok) * p.c.hkv + g.h) * p.group + rr - tok * p.group
                                      : ((size_t)blockIdx.x * 2 + (g.head ? 1 : 0)) * PRE_ROWS + threadIdx.x;
            *reinterpret_cast<float2 *>((g.whole ? p.row_ml : p.pre_ml) + to * 2) = make_float2(big, sum);
            s.to[threadIdx.x] = (g.whole ? p.row_o : p.pre_o) + to * D;
        }
#pragma unroll
        for (int c = 0; c < D; c += 32) {
            uint32_t r[32];
            pre_ld(o_addr + c, r);
            pre_wait_ld();
            float4 *mine = reinterpret_cast<float4 *>(s.merge + threadIdx.x * LD);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const auto o = [&](int j) { return last >= 0 ? __uint_as_float(r[4 * i + j]) * part * part : 0.f; };
                mine[i] = make_float4(o(0), o(1), o(2), o(3));
            }
            pre_bar();
            for (int e = threadIdx.x; e < rows * 8; e += 256) {
                const float *from = s.merge + (e / 8) * LD + e % 8 * 4;
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
                for (int i = 0; i < parts; ++i) {
                    const float4 y = *reinterpret_cast<const float4 *>(from + i * each * LD);
                    sum.x += y.x, sum.y += y.y, sum.z += y.z, sum.w += y.w;
                }
                *reinterpret_cast<float4 *>(s.to[e / 8] + c + e % 8 * 4) = sum;
            }
            pre_bar();
        }
        pre_fence_before();
    }
}

template <int D, int P>
__global__ void __launch_bounds__(PRE_THREADS, 1) cache_prefix_kernel(const AttParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    const PreShared s = pre_shared<D, P>(p);
    const int tid = threadIdx.x, warp = __shfl_sync(FULL, tid / 32, 0);
    if (tid == 0) *s.total = 0;
    const AttSeq seq = att_groups<P>(p, s.groups, false);
    att_others<P, ATT_GROUPS>(p, s.groups, seq, s.total);
    for (int g = tid; g < p.ngroups; g += PRE_THREADS) {
        const AttSeq q = att_unit<P, ATT_GROUPS>(p, s.groups, g, false);
        s.unit[g] = make_int4(q.q0, q.cnt, q.hi, s.groups.lead[g]);
        s.prefix[g + 1] = pre_items(p, q.cnt, q.hi);
    }
    if (tid < p.ring) {
        mbar_init(&s.full[tid], 1);
        mbar_init(&s.empty[tid], 8);
    }
    if (tid == 64) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&s.s_ready[x], 8);
            mbar_init(&s.s_done[x], 1);
            mbar_init(&s.o_ready[x], 8);
            mbar_init(&s.o_done[x], 1);
        }
        mbar_init(s.q_full, 4);
        mbar_init(s.q_empty, 1);
        mbar_init(s.drain, 1);
        s.ctrl[0] = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    att_running(s.prefix, p.ngroups);
    const int ctas = att_share(p, s.prefix[p.ngroups], (long long)*s.total);
    if ((int)blockIdx.x >= ctas) return;
    if (tid == 0) s.ctrl[2] = ctas;
    if (warp == PRE_ISSUER) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(saddr(&s.ctrl[1])) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        pre_fence_before();
    }
    __syncthreads();
    pre_fence_after();
    const uint32_t tmem = (uint32_t)s.ctrl[1];
    if ((saddr(s.tiles) & 1023) != 0) {
        if (tid == 0) note_failure(p.c.status, MK_ERR_DEVICE_CHECK, -1, -2, -1);
    } else if (warp < 8) {
        pre_rows<D, P>(p, s, tmem);
    } else if (warp < 12) {
        pre_convert<D, P, false>(p, s);
    } else if (warp < 16) {
        pre_convert<D, P, true>(p, s);
    } else if (warp == 16) {
        pre_produce<D, P>(p, s);
    } else if (warp == PRE_ISSUER) {
        pre_products<D, P>(p, s, tmem);
    }
    __syncwarp();
    __syncthreads();
    if (warp == PRE_ISSUER) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

int prefix_launch(const mk_cache_desc *cache, AttParams &p, cudaStream_t stream) {
    const int D = cache->head_dim, P = cache->page_tokens;
    const int fixed = pre_fixed_bytes(p.ngroups) + 4 * P * D * 2;
    p.ring = std::min(PRE_MAXRING, (SERVE_SMEM - fixed) / (2 * P * D));
    const int smem = fixed + p.ring * 2 * P * D;
    void (*f)(const AttParams) = D == 64 ? (P == 32 ? cache_prefix_kernel<64, 32> : cache_prefix_kernel<64, 64>)
                                         : (P == 32 ? cache_prefix_kernel<128, 32> : cache_prefix_kernel<128, 64>);
    static std::atomic<uint32_t> ready[SERVE_MAX_DEVICES];
    if (int rc = serve_prepare(reinterpret_cast<const void *>(f), ready, (D == 128 ? 2 : 0) + (P == 64 ? 1 : 0), false)) return rc;
    f<<<p.sms, PRE_THREADS, smem, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MK_OK : serve_cuda_fail(e, "prefix attention launch");
}

}  // namespace mk
