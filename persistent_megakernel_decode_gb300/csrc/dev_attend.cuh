// Shared by the cache attention's kernels (attend.cu, prefix.cu): parameters,
// what a sequence or a group of sequences asks for, work items cut into ranges.
#pragma once
#include <algorithm>
#include <climits>

#include "dev_serve.cuh"

namespace mk {

constexpr int ATT_MAXB = 1024;  // sequences per call

struct AttParams {
    CacheView c;  // of the layer: k, v, ks, vs point at it
    const uint16_t *q;
    uint16_t *out;
    float *lse;
    int64_t qs_t, qs_h, os_t, os_h;
    const int *table, *lens, *q_start;
    int batch, width, group, tokens, max_tokens, window, sinks, sink_pages, ring, ctas;
    float scale_log2;
    // workspace: partial (m, l) [ctas][2][RT][2]; partial O [ctas][2][RT][D]
    float *part_ml, *part_o;
    // shared prefixes: groups of consecutive sequences; what a row's own tokens
    // and its group's give, where one CTA had all of it: (m, l) [2][tokens][q
    // heads][2], O [2][tokens][q heads][D]
    const int *groups, *shared;
    int ngroups;
    float *row_ml, *row_o;
    // The groups' pages are a launch of their own, on part of `sms` SMs: rows of
    // its tiles (PRE_ROWS: prefix.cu's, else attend.cu's; 0: there is none, every
    // sequence reads its pages) and of the other one's, and what its CTAs cut, like
    // part_ml and part_o.
    int sms, pre_rt, rt;
    float *pre_ml, *pre_o;
};

// ln of the sum of exponentials: maximum in log2 units, sum times 2^14.
DEV float att_lse(float big, float sum) {
    return sum == 0.f ? -INFINITY : (big - 14.f + log2f(sum)) * 0.6931471805599453f;
}
// 1 / the sum of exponentials, from their sum times 2^14.
DEV float att_inverse(float sum) { return sum == 0.f ? 0.f : 16384.f / sum; }

// The first position that a query at pos sees (pos < 0: sees none, any window's end fits 32 bits).
DEV int att_least(int pos, int window) { return window > 0 && pos >= window ? pos - window + 1 : 0; }

// What a sequence asks for: its query rows, and the pages that any row sees:
// [0, hi) without the `gap` pages behind those of the sinks.
struct AttSeq {
    int q0, cnt, len, gap, hi;
    bool bad;  // its rows are not known
};
// The page of a sequence's i-th seen one.
DEV int att_page(const AttParams &p, int i, int gap) { return i < p.sink_pages ? i : i + gap; }

template <int P>
DEV AttSeq att_seq(const AttParams &p, int b, bool report) {
    AttSeq s;
    s.bad = false;
    s.len = p.lens[b];
    s.q0 = p.q_start ? p.q_start[b] : b * p.max_tokens;
    s.cnt = (p.q_start ? p.q_start[b + 1] : s.q0 + p.max_tokens) - s.q0;
    if (s.q0 < 0 || s.cnt < 0 || s.q0 > p.tokens || s.cnt > p.tokens - s.q0) {  // its rows are not known: none
        if (report) note_failure(p.c.status, MK_ERR_DEVICE_CHECK, b, s.q0, -1);
        s.q0 = s.cnt = s.len = s.gap = s.hi = 0;
        s.bad = true;
        return s;
    }
    if (s.len < 0 || (int64_t)s.len > (int64_t)p.width * P) {
        if (report) note_failure(p.c.status, MK_ERR_DEVICE_CHECK, b, s.len, -1);
        s.len = 0;
    }
    s.hi = (s.len + P - 1) / P;
    const int64_t first = (int64_t)s.len - s.cnt - p.window + 1;
    const int lo = p.window > 0 && first > 0 ? min((int)(first / P), s.hi) : 0;
    s.gap = max(0, lo - p.sink_pages);
    return s;
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

// CTA of work item x when `total` items are cut into `ctas` <= total ranges [c total / ctas, (c + 1) total / ctas).
DEV int att_owner(long long x, long long total, int ctas) { return (int)att_div((x + 1) * ctas - 1, total); }

// Shared prefixes.  lim[g]: the pages that all rows of group g see and take
// together; lead[g]: the sequence whose table row names them.
struct AttGroups {
    int *lead, *lim, *grp;  // [ngroups], [ngroups], [ngroups + 1]: the groups' first sequences
};
__host__ __device__ constexpr int att_group_bytes(int n) { return n ? (3 * n + 1) * 4 : 0; }
DEV AttGroups att_groups_at(void *at, int n) {
    int *x = static_cast<int *>(at);
    return {x, x + n, x + 2 * n};
}
// The group of a sequence, or -1.
DEV int att_group_of(const AttParams &p, const AttGroups &s, int b) {
    int a = 0, z = p.ngroups;  // the last group that begins at or before b
    while (z - a > 1) {
        const int mid = (a + z) / 2;
        if (s.grp[mid] <= b) a = mid;
        else z = mid;
    }
    return b >= s.grp[a] && b < s.grp[a + 1] ? a : -1;
}
// By the whole block; returns sequence threadIdx.x (what fails there is reported
// here).  What `shared` says is a bound: only full pages, and of
// them those that every query of the group sees whole.
template <int P>
DEV AttSeq att_groups(const AttParams &p, const AttGroups &s, bool report) {
    const int n = p.ngroups, tid = threadIdx.x, threads = blockDim.x;
    // the first of everything at once: one round trip
    const AttSeq mine = tid < p.batch ? att_seq<P>(p, tid, report) : AttSeq{0, 0, 0, 0, 0, false};
    const int share = tid < n ? p.shared[tid] : 0;
    bool bad = false;
    for (int g = tid; g <= n; g += threads) {
        const int x = p.groups[g];
        s.grp[g] = x;
        bad |= x < 0 || x > p.batch || (g < n && p.groups[g + 1] < x);
    }
    bad = __syncthreads_or(bad);
    if (bad && report && tid == 0) note_failure(p.c.status, MK_ERR_DEVICE_CHECK, -1, -1, -1);
    for (int g = tid; g < n; g += threads) {
        const int x = g == tid ? share : p.shared[g];
        if (x < 0 && report) note_failure(p.c.status, MK_ERR_DEVICE_CHECK, s.grp[g], x, -1);
        s.lead[g] = INT_MAX;
        s.lim[g] = bad || !p.pre_rt || s.grp[g + 1] - s.grp[g] < 2 ? 0 : max(x, 0) / P;
    }
    __syncthreads();
    for (int b = tid; b < p.batch && !bad; b += threads) {
        const int g = att_group_of(p, s, b);
        if (g < 0) continue;
        const AttSeq q = b == tid ? mine : att_seq<P>(p, b, false);
        if (q.bad) atomicMin(&s.lim[g], 0);  // where its rows begin is not known either
        if (q.cnt == 0) continue;
        atomicMin(&s.lead[g], b);
        atomicMin(&s.lim[g], max(0, q.len - q.cnt + 1) / P);
    }
    __syncthreads();
    return mine;
}
// What a launch is for: sequences by themselves; with shared prefixes, sequences
// over the pages behind them; groups over the shared pages.
enum AttKind { ATT_PLAIN, ATT_OWN, ATT_GROUPS };
DEV int att_units(const AttParams &p, AttKind kind) { return kind == ATT_GROUPS ? p.ngroups : p.batch; }
// Unit v: a sequence (`mine`: what att_groups returned), or a group's rows over its pages (every row sees all).
template <int P, AttKind KIND>
DEV AttSeq att_unit(const AttParams &p, const AttGroups &s, int v, bool report, const AttSeq *mine = nullptr) {
    if constexpr (KIND == ATT_PLAIN) {
        return att_seq<P>(p, v, report);
    } else if constexpr (KIND == ATT_OWN) {
        AttSeq q = mine && v == (int)threadIdx.x ? *mine : att_seq<P>(p, v, report);
        const int g = att_group_of(p, s, v);
        q.gap = g < 0 ? 0 : min(s.lim[g], q.hi);
        return q;
    } else {
        AttSeq q{0, 0, 0, 0, 0, false};
        if (s.lim[v] > 0 && s.lead[v] < p.batch) {
            q.q0 = p.q_start ? p.q_start[s.grp[v]] : s.grp[v] * p.max_tokens;
            q.cnt = (p.q_start ? p.q_start[s.grp[v + 1]] : s.grp[v + 1] * p.max_tokens) - q.q0;
            q.hi = s.lim[v];
            q.len = q.hi * P;
        }
        return q;
    }
}

// Shared pages in a launch of their own (prefix.cu): tiles of 128 rows, and what
// a unit (group, tile, kv head) costs beside its pages, in pages.
constexpr int PRE_ROWS = 128, PRE_FIXED = 8;
DEV long long pre_items(const AttParams &p, int cnt, int np) {
    return np && cnt ? (long long)((cnt * p.group + PRE_ROWS - 1) / PRE_ROWS) * p.c.hkv * (np + PRE_FIXED) : 0;
}
DEV int pre_used(long long total, int ctas) { return (int)max(1ll, min((long long)ctas, total)); }


// Warps side by side on a tile of so many rows (tiles of rt rows, 8 or 16 a warp): 1, 2 or 4.
__host__ __device__ constexpr int att_side_of(int rt, int rows) {
    const int per = rt == 8 ? 8 : 16, need = ((rt < rows ? rt : rows) + per - 1) / per;
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
DEV long long att_items_of(const AttParams &p, int rt, int cnt, int np) {
    const int rows = cnt * p.group, tiles = (rows + rt - 1) / rt, fixed = att_fixed_items(rt);
    if (tiles == 0 || np <= 0) return 0;
    return p.c.hkv * ((tiles - 1) * ((long long)np * att_side_of(rt, rt) + fixed) +
                      (long long)np * att_side_of(rt, rows - (tiles - 1) * rt) + fixed);
}

// Work items of a group.
DEV long long att_group_items(const AttParams &p, int cnt, int np) {
    return np == 0 ? 0 : p.pre_rt == PRE_ROWS ? pre_items(p, cnt, np) : att_items_of(p, p.pre_rt, cnt, np);
}
// Both launches run beside each other, on SMs shared out by their work: the CTAs
// of the groups' one.  By the clock a page through prefix.cu's tiles takes an SM as
// long as 2.5 items of the sequences' launch, an item of attend.cu's for groups
// 1.3 (0.95 and 0.5 us; with heads of 128 and pages of 64, taken for others too).
DEV int att_share(const AttParams &p, long long groups, long long own) {
    if (groups == 0) return 0;
    if (own == 0) return p.sms;
    const long long a = groups * (p.pre_rt == PRE_ROWS ? 15 : 8), all = a + 6 * own;
    const long long n = (a * p.sms + all / 2) / all;
    return (int)min((long long)p.sms - 1, max(1ll, n));
}
// Sum of v over the block, in *to (zeroed before a barrier; read after one).
DEV void att_total(long long v, unsigned long long *to) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL, v, o);
    if (threadIdx.x % 32 == 0 && v) atomicAdd(to, (unsigned long long)v);
}
// The other launch's items, summed over the block.
template <int P, AttKind KIND>
DEV void att_others(const AttParams &p, const AttGroups &s, const AttSeq &mine, unsigned long long *to) {
    long long v = 0;
    if constexpr (KIND == ATT_GROUPS) {
        for (int b = threadIdx.x; b < p.batch; b += blockDim.x) {
            const AttSeq q = att_unit<P, ATT_OWN>(p, s, b, false, &mine);
            v += att_items_of(p, p.rt, q.cnt, q.hi - q.gap);
        }
    } else {
        for (int g = threadIdx.x; g < p.ngroups; g += blockDim.x) {
            const AttSeq q = att_unit<P, ATT_GROUPS>(p, s, g, false);
            v += att_group_items(p, q.cnt, q.hi);
        }
    }
    att_total(v, to);
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

int prefix_launch(const mk_cache_desc *cache, AttParams &p, cudaStream_t stream);  // prefix.cu

}  // namespace mk
