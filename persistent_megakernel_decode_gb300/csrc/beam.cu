// Beam search's selection: the best continuations over beams and vocabulary.
//
// Mathematics.  A candidate (beam w, token v) has the total s_w + z_wv -
// log sum_v exp z_wv; the `num` largest of a prompt's beams are wanted, ties to
// the lowest w V + v.  Within a beam the order is that of the logits, so each
// beam's row gives its `num` largest logits and the sum of its exponentials,
// and the beams' short sorted lists are merged by their totals.
//
// The order between beams hangs on the sums: two totals closer than their
// errors would change places.  Totals are therefore formed in 64 bits, and the
// sum is kept to a few 2^-30 of itself: the row's largest logits (where single
// rounding errors weigh) by the fixed-point weights of dev_weigh.cuh, the rest
// as fp32 2^f after a two-part reduction of the argument, whose errors (2^-23
// of a term, either way) average out; all partial sums are joined as integers,
// so no order of arrival changes anything.
//
// The largest of a row without sorting it: a bound that at least `num` threads'
// largest values reach is found by bisection, one barrier and vote a step; the
// few logits that reach it (at most as many per thread as it holds) are ranked
// by comparing each with all.  Ties at the bound go on by bisection over the
// index.
//
// Work split.  One cluster of CTAs per row, the row's logits in registers; the
// clusters' lists meet in their first CTA.  A second, dependent launch merges
// the beams of a prompt.  Bytes bound it: each logit is read once.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>

#include "dev_weigh.cuh"

namespace cg = cooperative_groups;

namespace mk {

constexpr int BM_THREADS = 512, BM_WARPS = BM_THREADS / 32;
constexpr int BM_MAXCTAS = 16, BM_MAXPER = 80;  // CTAs per row, logits per thread
constexpr int BM_MAXVOCAB = 622592;
constexpr int BM_MAXBEAMS = 64, BM_MAXNUM = 128;

// What the second launch needs of a row beside its list.
struct BeamRow {
    float top;              // the largest logit
    int ref;                // `rest` is in units of 2^(ref - 44)
    unsigned long long list, rest;  // sums: of the weights relative to the largest, in 2^-44; of the others
};

struct BeamParams {
    const void *logits;
    int64_t row_stride;
    int vocab, beams, num, chunk, ctas, cap;
    const float *scores;
    const uint8_t *finished;
    int end;
    BeamRow *rows;              // workspace: [batch x beams]
    unsigned long long *keys;   // workspace: [batch x beams][num], ascending, then KEY_NONE
    float *out;
    int *parents, *tokens;
};

struct alignas(16) BeamShared {  // the lists lie behind it
    uint32_t table[32];
    uint32_t tops[BM_MAXCTAS];                       // every CTA's largest logit, ordered
    unsigned long long list[BM_MAXCTAS], rest[BM_MAXCTAS];  // every CTA's sums
    unsigned long long red[2][BM_WARPS];
    uint32_t red_u[BM_WARPS];
    int count;
};

// A beam that is extended: its score is finite and it has not finished.
DEV bool beam_live(const BeamParams &p, int64_t row) {
    const float s = p.scores[row];
    return fabsf(s) < INFINITY && !(p.finished && p.finished[row]);
}

// One logit: NaN counts as -inf, -0 as +0 (they are equal: the index decides).
DEV float beam_logit(float x) { return fmaxf(x, -INFINITY) + 0.f; }

DEV float key_value(unsigned long long key) {
    const uint32_t o = ~(uint32_t)(key >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}

DEV void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
DEV void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

DEV float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

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

// Ranks of `n` lists' entries among all of them: lists[l][0 .. len(l)) ascend
// by `better`, and each entry's rank is its place plus, for every other list,
// how many of that come before it.  rank[l * stride + i] must be zeroed.
template <typename Len, typename Before>
DEV void merge_ranks(int n, int stride, const Len &len, const Before &before, int *rank) {
    const int pairs = n * n * stride;
    for (int x = threadIdx.x; x < pairs; x += BM_THREADS) {
        const int other = x % n, e = x / n, l = e / stride, i = e % stride;
        if (i >= len(l)) continue;
        int a = 0, z = len(other);
        if (other == l) {
            a = i;
        } else {  // the first of `other` that does not come before
            while (a < z) {
                const int mid = (a + z) / 2;
                if (before(other, mid, l, i)) a = mid + 1;
                else z = mid;
            }
        }
        if (a) atomicAdd(&rank[e], a);
    }
}

template <int E, bool BF16>
__global__ void __launch_bounds__(BM_THREADS) beam_row_kernel(const BeamParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    constexpr int VEC = BF16 ? 8 : 4;
    BeamShared &s = *reinterpret_cast<BeamShared *>(mk_smem);
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int rank = (int)(blockIdx.x % p.ctas);
    const int64_t row = blockIdx.x / p.ctas;
    if (!beam_live(p, row)) return;  // the whole cluster
    cluster_arrive();
    cg::cluster_group cl = cg::this_cluster();
    // behind s: candidates [cap], all CTAs' lists [ctas][num], ranks of either
    unsigned long long *cand = reinterpret_cast<unsigned long long *>(mk_smem + sizeof(BeamShared));
    unsigned long long *lists = cand + p.cap;
    int *ranks = reinterpret_cast<int *>(lists + p.ctas * p.num);

    // the CTA's logits [first, last), VEC of a thread together, from the 16-byte boundary at or before the first
    const int first = min(rank * p.chunk, p.vocab), last = min(first + p.chunk, p.vocab);
    constexpr int SIZE = BF16 ? 2 : 4;
    const char *base = static_cast<const char *>(p.logits) + row * p.row_stride * SIZE;
    const int shift = (int)(((uintptr_t)base + (size_t)first * SIZE) % 16 / SIZE);
    const auto at = [&](int i) { return first - shift + (i / VEC * BM_THREADS + tid) * VEC + i % VEC; };
    float v[E];
#pragma unroll
    for (int i = 0; i < E; i += VEC) {
        const int x = at(i);
        if (x >= first && x + VEC <= last) {
            const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(base + (size_t)x * SIZE));
            if constexpr (BF16) {
                float f[8];
                bf16x8(w, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i + j] = f[j];
            } else {
                v[i] = __uint_as_float(w.x), v[i + 1] = __uint_as_float(w.y);
                v[i + 2] = __uint_as_float(w.z), v[i + 3] = __uint_as_float(w.w);
            }
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                v[i + j] = -INFINITY;
                if (x + j >= first && x + j < last) {
                    if constexpr (BF16) v[i + j] = bf16_at(reinterpret_cast<const uint16_t *>(base), x + j);
                    else v[i + j] = reinterpret_cast<const float *>(base)[x + j];
                }
            }
        }
    }
    if (tid < 32) s.table[tid] = c_table[tid];
    if (tid == 0) s.count = 0;
    for (int i = tid; i < p.cap; i += BM_THREADS) ranks[i] = 0;
    float most = -INFINITY;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        v[i] = beam_logit(v[i]);
        most = fmaxf(most, v[i]);
    }
    const uint32_t mine = ordered_bits(most);
    uint32_t top_bits = __reduce_max_sync(FULL, mine);
    if (lane == 0) s.red_u[warp] = top_bits;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < BM_WARPS; ++i) top_bits = max(top_bits, s.red_u[i]);
    cluster_wait();  // every CTA runs: its shared memory may be written
    if (tid < p.ctas) *cl.map_shared_rank(&s.tops[rank], tid) = top_bits;
    cluster_arrive();

    // a bound that num threads' largest reach, and so many at most that their logits fit the list
    const int limit = p.cap / E;
    uint32_t lo = 0x00800000u, hi = top_bits;  // from the least value above -inf
    int upto = INT_MAX;                        // of the logits at the bound, those up to this index
    if (__syncthreads_count(mine >= lo) > limit) {
        bool found = false;
        while (lo < hi) {
            const uint32_t mid = lo + (hi - lo + 1) / 2;
            const int n = __syncthreads_count(mine >= mid);
            if (n > limit) {
                lo = mid;
            } else if (n >= p.num) {
                lo = mid;
                found = true;
                break;
            } else {
                hi = mid - 1;
            }
        }
        if (!found) {  // many threads have the same largest logit
            const float bound = key_value((unsigned long long)~lo << 32);
            uint32_t more = 0;
#pragma unroll
            for (int i = 0; i < E; ++i) more += v[i] > bound;
            const int need = p.num - (int)block_sum(more, s.red_u);
            int a = first - 1, z = last - 1;  // the least index up to which `need` logits are at the bound
            if (need <= 0) z = a;
            while (z - a > 1) {
                const int mid = a + (z - a) / 2;
                uint32_t n = 0;
#pragma unroll
                for (int i = 0; i < E; ++i) n += v[i] == bound && at(i) <= mid;
                if ((int)block_sum(n, s.red_u) >= need) z = mid;
                else a = mid;
            }
            upto = z;
        }
    }
    const float bound = key_value((unsigned long long)~lo << 32);
    const auto listed = [&](float x, int i) { return x > bound || (x == bound && i <= upto); };
    if (mine >= lo) {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (listed(v[i], at(i))) cand[atomicAdd(&s.count, 1)] = sample_key(v[i], at(i));
    }
    __syncthreads();
    const int n = s.count, kept = min(n, p.num);
    // ranks: the threads of a column share a candidate
    int wide = 32;
    while (wide < n && wide < BM_THREADS) wide *= 2;
    for (int i = tid % wide; i < n; i += wide) {
        const unsigned long long key = cand[i];
        int before = 0;
        for (int j = tid / wide; j < n; j += BM_THREADS / wide) before += cand[j] < key;
        if (before) atomicAdd(&ranks[i], before);
    }
    cluster_wait();  // the largest logits of all CTAs
    uint32_t row_top = 0;
    for (int i = 0; i < p.ctas; ++i) row_top = max(row_top, s.tops[i]);
    const float top = key_value((unsigned long long)~row_top << 32);
    const Weigher weigh{top, 1.44269502162933349609375f, 1.92596303350011e-08f, s.table};
    unsigned long long list = 0, rest = 0;
    int ref = 0;
    if (top > -INFINITY) {
        if (fabsf(top) <= 1e5f) {
            // 2^(x log2(e) - ref): x log2(e) = n + f, f good to 2^-26 (the largest sum per thread is E)
            constexpr float ROUND = 12582912.f;
            const float least = top - 80.f;  // e^-80: nothing beside 2^-44
            ref = (int)ceilf(top * weigh.ch);
            float a[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float x = fmaxf(v[i], least);
                const float t = fmaf(x, weigh.ch, ROUND), k = t - ROUND;
                const float f = fmaf(x, weigh.cl, fmaf(x, weigh.ch, -k));
                const float e = __int_as_float(__float_as_int(exp2_approx(f)) + ((__float_as_int(t) - __float_as_int(ROUND) - ref) << 23));
                a[i % 2] += listed(v[i], at(i)) || v[i] == -INFINITY ? 0.f : e;
            }
            rest = __float2ull_rn((a[0] + a[1]) * 0x1p44f);
            for (int i = tid; i < n; i += BM_THREADS) list += weigh(key_value(cand[i]));
        } else {
            for (int i = 0; i < E; ++i) list += v[i] == -INFINITY ? 0 : weigh(v[i]);
        }
    }
    list = warp_sum64(list);
    rest = warp_sum64(rest);
    if (lane == 0) {
        s.red[0][warp] = list;
        s.red[1][warp] = rest;
    }
    __syncthreads();  // the ranks too
    unsigned long long *to = cl.map_shared_rank(lists, 0) + rank * p.num;
    for (int i = tid; i < n; i += BM_THREADS)
        if (ranks[i] < p.num) to[ranks[i]] = cand[i];
    for (int i = kept + tid; i < p.num; i += BM_THREADS) to[i] = KEY_NONE;
    if (tid < 2) {
        unsigned long long sum = 0;
        for (int i = 0; i < BM_WARPS; ++i) sum += s.red[tid][i];
        *cl.map_shared_rank(tid ? &s.rest[rank] : &s.list[rank], 0) = sum;
    }
    cluster_arrive();
    cluster_wait();
    if (rank != 0) return;

    // the CTAs' lists into one
    for (int i = tid; i < p.ctas * p.num; i += BM_THREADS) ranks[i] = 0;
    __syncthreads();
    const auto len = [&](int) { return p.num; };
    merge_ranks(p.ctas, p.num, len, [&](int l, int i, int m, int j) {  // KEY_NONE: among themselves in the lists' order
        const unsigned long long x = lists[l * p.num + i], y = lists[m * p.num + j];
        return x < y || (x == y && l < m);
    }, ranks);
    __syncthreads();
    for (int i = tid; i < p.ctas * p.num; i += BM_THREADS)
        if (ranks[i] < p.num) p.keys[row * p.num + ranks[i]] = lists[i];
    if (tid == 0) {
        BeamRow r{top, ref, 0, 0};
        for (int i = 0; i < p.ctas; ++i) {
            r.list += s.list[i];
            r.rest += s.rest[i];
        }
        p.rows[row] = r;
    }
}

// fp64 totals as integers that rise with them.
DEV unsigned long long ordered64(double x) {
    const long long b = __double_as_longlong(x + 0.0);
    return b < 0 ? ~(unsigned long long)b : (unsigned long long)b | 0x8000000000000000ull;
}

// One CTA per prompt: the beams' lists into one, by their totals.
__global__ void __launch_bounds__(BM_THREADS) beam_merge_kernel(const BeamParams p) {
    double *s_log = reinterpret_cast<double *>(mk_smem);  // [64]: of the sum of exp(z - top)
    int *s_len = reinterpret_cast<int *>(s_log + BM_MAXBEAMS);  // [64]
    const int tid = threadIdx.x, W = p.beams, K = p.num;
    unsigned long long *total = reinterpret_cast<unsigned long long *>(s_len + BM_MAXBEAMS);  // [W][K]
    int *token = reinterpret_cast<int *>(total + W * K), *ranks = token + W * K;
    const int64_t row0 = (int64_t)blockIdx.x * W;
    for (int i = tid; i < W * K; i += BM_THREADS) ranks[i] = 0;
    if (tid < W) s_len[tid] = 0;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid < W && beam_live(p, row0 + tid)) {
        const BeamRow r = p.rows[row0 + tid];
        double sum = (double)r.list;
        if (r.rest) sum += (double)r.rest * exp2((double)r.ref - (double)r.top * 1.4426950408889634);
        s_log[tid] = log(sum * 0x1p-44);
    }
    __syncthreads();
    for (int i = tid; i < W * K; i += BM_THREADS) {
        const int w = i / K, j = i % K;
        const float score = p.scores[row0 + w];
        double t = -INFINITY;
        int v = -1;
        if (beam_live(p, row0 + w)) {
            const unsigned long long key = p.keys[(row0 + w) * K + j];
            if (key != KEY_NONE) {
                const float z = key_value(key), top = p.rows[row0 + w].top;
                t = (double)score + ((z == top ? 0.0 : (double)z - (double)top) - s_log[w]);
                v = (int)(uint32_t)key;
            }
        } else if (j == 0 && fabsf(score) < INFINITY) {  // finished: goes on as it is
            t = score;
            v = p.end;
        }
        total[i] = ordered64(t);
        token[i] = v;
        if (t > -INFINITY) atomicAdd(&s_len[w], 1);  // they come first
    }
    __syncthreads();
    // Of equal totals the lower beam comes first; a beam's own have their order.
    merge_ranks(W, K, [&](int l) { return s_len[l]; }, [&](int l, int i, int m, int j) {
        const unsigned long long x = total[l * K + i], y = total[m * K + j];
        return x > y || (x == y && l < m);
    }, ranks);
    __syncthreads();
    int all = 0;
    for (int w = 0; w < W; ++w) all += s_len[w];
    for (int i = tid; i < W * K; i += BM_THREADS) {
        const int w = i / K;
        if (i % K >= s_len[w] || ranks[i] >= K) continue;
        const int64_t to = (int64_t)blockIdx.x * K + ranks[i];
        const unsigned long long o = total[i];
        p.out[to] = (float)__longlong_as_double(o >> 63 ? o & 0x7fffffffffffffffull : ~o);
        p.parents[to] = w;
        p.tokens[to] = token[i];
    }
    for (int i = all + tid; i < K; i += BM_THREADS) {
        const int64_t to = (int64_t)blockIdx.x * K + i;
        p.out[to] = -INFINITY;
        p.parents[to] = p.tokens[to] = -1;
    }
}

using BeamFn = void (*)(const BeamParams);
static constexpr int BM_PER[] = {8, 16, 24, 32, 48, BM_MAXPER};
template <bool BF16>
static BeamFn beam_kernel(int i) {
    return i == 0 ? beam_row_kernel<8, BF16> : i == 1 ? beam_row_kernel<16, BF16> : i == 2 ? beam_row_kernel<24, BF16>
         : i == 3 ? beam_row_kernel<32, BF16> : i == 4 ? beam_row_kernel<48, BF16> : beam_row_kernel<BM_MAXPER, BF16>;
}

static int beam_sizes(const mk_beam_desc *d) {
    if (!d) return set_error(MK_ERR_INVALID, "null descriptor");
    if (d->batch < 0 || d->beams <= 0 || d->num <= 0 || d->vocab <= 0)
        return set_error(MK_ERR_INVALID, "batch negative, or beams, num or vocab not positive");
    if (d->beams > BM_MAXBEAMS || d->num > BM_MAXNUM) return set_error(MK_ERR_UNSUPPORTED, "more than 64 beams or 128 continuations");
    if (d->vocab > BM_MAXVOCAB) return set_error(MK_ERR_UNSUPPORTED, "vocab above 622592");
    if ((int64_t)d->batch * d->beams > INT32_MAX / BM_MAXCTAS) return set_error(MK_ERR_UNSUPPORTED, "too many rows");
    return MK_OK;
}
static uint64_t beam_row_bytes(const mk_beam_desc *d) { return (uint64_t)d->batch * d->beams * sizeof(BeamRow); }

}  // namespace mk

using namespace mk;

extern "C" {

int mk_beam_select_workspace(const mk_beam_desc *d, uint64_t *bytes) {
    if (!bytes) return set_error(MK_ERR_INVALID, "bytes is null");
    if (int rc = beam_sizes(d)) return rc;
    *bytes = beam_row_bytes(d) + (uint64_t)d->batch * d->beams * d->num * 8;
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
    p.rows = static_cast<BeamRow *>(workspace);
    p.keys = reinterpret_cast<unsigned long long *>(static_cast<uint8_t *>(workspace) + beam_row_bytes(d));
    p.out = reinterpret_cast<float *>(d->out_scores);
    p.parents = reinterpret_cast<int *>(d->parents);
    p.tokens = reinterpret_cast<int *>(d->tokens);
    p.ctas = rows <= 64 ? 16 : 8;
    while (p.ctas > 1 && d->vocab < p.ctas * 1024) p.ctas /= 2;
    const int vec = d->bf16 ? 8 : 4;
    const auto chunk_of = [&](int ctas) { return ((d->vocab + ctas - 1) / ctas + vec - 1) / vec * vec; };
    while (p.ctas < BM_MAXCTAS && chunk_of(p.ctas) + vec > BM_MAXPER * BM_THREADS) p.ctas *= 2;
    p.chunk = chunk_of(p.ctas);
    int per = 0;
    while (p.chunk + vec > BM_PER[per] * BM_THREADS) ++per;
    // the list holds all logits of as many threads as may reach the bound
    p.cap = std::max(64, 2 * p.num) * BM_PER[per];
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    BeamFn f = d->bf16 ? beam_kernel<true>(per) : beam_kernel<false>(per);
    static std::atomic<uint32_t> ready[SERVE_MAX_DEVICES];
    if (int rc = serve_prepare(reinterpret_cast<const void *>(f), ready, 2 * per + (d->bf16 ? 1 : 0), true)) return rc;
    if (int rc = serve_prepare(reinterpret_cast<const void *>(beam_merge_kernel), ready, 31, false)) return rc;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = p.ctas;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(rows * p.ctas));
    cfg.blockDim = dim3(BM_THREADS);
    cfg.dynamicSmemBytes = sizeof(BeamShared) + p.cap * 8 + p.ctas * p.num * 8 + std::max(p.cap, p.ctas * p.num) * 4;
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, f, (const BeamParams)p);
    if (e != cudaSuccess) return serve_cuda_fail(e, "beam selection launch");
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)d->batch);
    cfg.dynamicSmemBytes = BM_MAXBEAMS * 12 + p.beams * p.num * 16;
    e = cudaLaunchKernelEx(&cfg, beam_merge_kernel, (const BeamParams)p);
    return e == cudaSuccess ? MK_OK : serve_cuda_fail(e, "beam merge launch");
}

}  // extern "C"
