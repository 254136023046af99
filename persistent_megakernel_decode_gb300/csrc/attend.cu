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
// (2^-8).  tcgen05 is not used here: its tiles take 64 rows or more of an
// operand from shared memory, a decode step has 4 to 16, and scores would cross
// tensor memory between the two products; bytes bound a decode step either way.
// (prefix.cu uses it, for the pages that large groups of sequences share.)
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
// CTA (one CTA per SM): ragged batches and single long sequences balance alike.
// A producer warp streams the pages through a shared-memory ring with bulk
// copies; the consumer warps take them in turn (as many side by side as the
// tile's rows need) and merge in shared memory.  A page that a tile does not
// see, or whose number is out of range, takes its turn in the ring without
// being loaded.  A slot is released behind a proxy fence (att_reads_done).  With sinks, a unit's pages are those of the sinks and those
// from the window's first on; the pages between are no items at all.
// A unit that one CTA covers is written at once; ranges cut by a CTA boundary
// go to the workspace and a second small launch (dependent launch, so that its
// start overlaps) merges them in order: results do not depend on timing.
//
// Shared prefixes.  Groups' shared pages are units of one launch (the page
// kernel's tiles, or prefix.cu's), what sequences have behind them are units of
// another, and the merge joins both.  The two run beside each other, on SMs that
// the device shares out by the items of each at their measured costs
// (dev_attend.cuh); an own part is short, so two CTAs of four warps take them on
// an SM (64 sequences of 16,000 shared tokens and 100-2,000 of their own: 82 us
// when that was chosen, with one CTA of eight warps 85, now 77; 4 x 8 beams: 43.7
// and 45).
//
// Measured (one GB300, device time): 16 sequences of 16-32K tokens, 32 q / 8
// kv heads of 128: 125 us, 6.3 TB/s, 93 % of the copy rate; 8 sequences of
// 512-4096, heads of 64: 13.5 us, of which the bytes are 2.8
// (two launches, two dependent look-ups, the ramp of the loads and the merge
// are the rest); 64 new tokens a sequence over 4000: 190 TFLOP/s, bound by the
// instructions per product that a 16-row operand held in registers costs; a
// prompt of 2048 new tokens: 377 us, 91 TFLOP/s, half of its tiles' pages
// passing through the ring unseen.
#include "dev_attend_pages.cuh"

namespace mk {

struct AttPlan {
    int rt, ctas, sms, pre_rt;  // pre_rt: rows of the groups' tiles
    uint64_t ml_bytes, o_bytes, row_ml_bytes, row_o_bytes, pre_ml_bytes, pre_o_bytes;
    uint64_t bytes() const { return ml_bytes + o_bytes + row_ml_bytes + row_o_bytes + pre_ml_bytes + pre_o_bytes; }
};

// Tiles of 8, 16, 32 or 64 rows: the least that takes so many.
static int att_tile(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }
// Rows of an average group and kv head from which prefix.cu's tiles are taken for
// its shared pages.  64 sequences (256 rows) behind 16,000 tokens: 82 us, with
// attend.cu's 120; 21 with drafted tokens in 3 groups (56 rows) 35 and 39; 4 x 8
// beams (32 rows) 46 and 44.  (Between 32 and 56 rows nothing was measured.)
constexpr int PRE_LEAST = 48;
// Pages of all sequences and kv heads, per SM, up to which nothing is shared: a
// launch more costs as much as reading so few again.  4 beams of a prompt of 300
// tokens (88 pages): 11 us, shared 16.  (The one such call measured.)
constexpr int ALONE_PAGES = 4;

// ngroups: 0 without shared prefixes
static int att_plan(const mk_cache_desc *c, const mk_attend_desc *a, int ngroups, AttPlan &pl) {
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
    const int group = a->q_heads / c->kv_heads;
    pl.rt = att_tile((int64_t)std::max(1, std::min(a->max_tokens, a->tokens)) * group);
    pl.pre_rt = 0;
    if (ngroups) {
        const int64_t rows = ((int64_t)a->tokens + ngroups - 1) / ngroups * group;  // of an average group
        const bool alone = (int64_t)a->batch * a->table_width * c->kv_heads <= (int64_t)ALONE_PAGES * sms;
        pl.pre_rt = alone ? 0 : rows >= PRE_LEAST ? PRE_ROWS : att_tile(rows);
        sms = std::max(sms, 2);  // both launches share them
    }
    pl.sms = sms;
    // no more CTAs than pages there can be (all tiles' together, each as many items as it has warps side by side)
    const int64_t side = pl.rt == 64 ? 4 : pl.rt == 32 ? 2 : 1;
    const int64_t tiles = a->batch + (int64_t)a->tokens * group / pl.rt;
    const int64_t items = std::min<int64_t>(tiles * c->kv_heads, INT32_MAX) * (a->table_width * side + att_fixed_items(pl.rt));
    pl.ctas = (int)std::min<int64_t>(ngroups ? 2 * sms : sms, std::max<int64_t>(1, items));
    pl.ml_bytes = ((uint64_t)pl.ctas * 2 * pl.rt * 8 + 255) / 256 * 256;
    pl.o_bytes = (uint64_t)pl.ctas * 2 * pl.rt * c->head_dim * 4;
    const uint64_t row_parts = ngroups ? 2ull * a->tokens * a->q_heads : 0;
    pl.row_ml_bytes = (row_parts * 8 + 255) / 256 * 256;
    pl.row_o_bytes = row_parts * c->head_dim * 4;
    pl.pre_ml_bytes = ((uint64_t)sms * 2 * pl.pre_rt * 8 + 255) / 256 * 256;
    pl.pre_o_bytes = (uint64_t)sms * 2 * pl.pre_rt * c->head_dim * 4;
    return MK_OK;
}

// One launch of the kernel over `units` units, its tiles of rt rows.
static int att_start(const mk_cache_desc *cache, AttParams &p, AttKind kind, int rt, int ctas, int units, bool after, cudaStream_t st) {
    const int D = cache->head_dim, P = cache->page_tokens;
    const int fixed = att_fixed_bytes(D, att_nt(rt), att_warps(kind)) + att_seq_bytes(units, p.ngroups) + 128;
    const int smem = kind == ATT_OWN ? SERVE_SMEM / 2 - 512 : SERVE_SMEM;  // (a CTA takes 1024 bytes more)
    p.ring = std::min(ATT_MAXRING, (smem - fixed) / (2 * P * D));
    p.ctas = ctas;
    const AttFn f = kind == ATT_PLAIN ? att_kernel_of<ATT_PLAIN>(D, P, rt) : att_shared_kernel(kind, D, P, rt);
    static std::atomic<uint32_t> ready[3][SERVE_MAX_DEVICES];
    const int variant = (D == 128 ? 8 : 0) + (P == 64 ? 4 : 0) + (rt == 8 ? 0 : rt == 16 ? 1 : rt == 32 ? 2 : 3);
    if (int rc = serve_prepare(reinterpret_cast<const void *>(f), ready[kind], variant, false)) return rc;
    cudaLaunchAttribute dep{};
    dep.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    dep.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(att_threads(kind, rt));
    cfg.dynamicSmemBytes = fixed + p.ring * 2 * P * D;
    cfg.stream = st;
    cfg.attrs = &dep;
    cfg.numAttrs = after ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, f, (const AttParams)p);
    return e == cudaSuccess ? MK_OK : serve_cuda_fail(e, "attention launch");
}

// share: null without shared prefixes
static int att_launch(const mk_cache_desc *cache, int layer, const mk_attend_desc *a, const mk_shared_desc *share,
                      void *workspace, uint64_t workspace_bytes, void *stream) {
    AttParams p{};
    AttPlan pl;
    if (int rc = cache_check(cache, p.c)) return rc;
    const int ngroups = share ? share->groups : 0;
    if (int rc = att_plan(cache, a, ngroups, pl)) return rc;
    if (layer < 0 || layer >= cache->layers) return set_error(MK_ERR_INVALID, "layer out of range");
    if (a->window < 0 || a->sinks < 0 || !(a->scale >= 0.f) || a->scale > 3e38f)
        return set_error(MK_ERR_INVALID, "window and sinks must not be negative, scale finite and not negative");
    if (a->batch == 0 || a->tokens == 0) return MK_OK;
    if (!a->q || !a->out || !a->table || !a->lens) return set_error(MK_ERR_INVALID, "null argument");
    if (a->q % 16 || a->out % 16 || a->lse % 4) return set_error(MK_ERR_INVALID, "q and out must be 16-byte aligned");
    for (int i = 0; i < 2; ++i)
        if (a->q_stride[i] % 8 || a->out_stride[i] % 8)
            return set_error(MK_ERR_INVALID, "q and out strides must be multiples of 8 elements");
    if (!workspace || (uintptr_t)workspace % 16 || workspace_bytes < pl.bytes())
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
    p.sinks = a->window ? std::min(a->sinks, a->table_width * P) : 0;
    p.sink_pages = p.sinks ? (p.sinks - 1) / P + 1 : 0;
    p.scale_log2 = a->scale * 1.4426950408889634f;
    p.rt = pl.rt;
    p.sms = pl.sms;
    p.pre_rt = pl.pre_rt;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.part_ml = reinterpret_cast<float *>(ws);
    p.part_o = reinterpret_cast<float *>(ws + pl.ml_bytes);
    if (ngroups) {
        p.groups = reinterpret_cast<const int *>(share->first);
        p.shared = reinterpret_cast<const int *>(share->shared);
        p.ngroups = ngroups;
        p.row_ml = reinterpret_cast<float *>(ws + pl.ml_bytes + pl.o_bytes);
        uint8_t *at = ws + pl.ml_bytes + pl.o_bytes + pl.row_ml_bytes;
        p.row_o = reinterpret_cast<float *>(at);
        at += pl.row_o_bytes;
        p.pre_ml = reinterpret_cast<float *>(at);
        p.pre_o = reinterpret_cast<float *>(at + pl.pre_ml_bytes);
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (pl.pre_rt) {
        const int rc = pl.pre_rt == PRE_ROWS ? prefix_launch(cache, p, st)
                                             : att_start(cache, p, ATT_GROUPS, pl.pre_rt, pl.sms, ngroups, false, st);
        if (rc) return rc;
    }
    // (with groups: on the SMs that their launch leaves)
    if (int rc = att_start(cache, p, ngroups ? ATT_OWN : ATT_PLAIN, pl.rt, pl.ctas, p.batch, pl.pre_rt > 0, st)) return rc;
    cudaLaunchAttribute dep{};
    dep.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    dep.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(((int64_t)p.tokens * a->q_heads + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = &dep;
    cfg.numAttrs = 1;
    cfg.dynamicSmemBytes = (size_t)(p.batch + 1) * 8 + (att_group_bytes(ngroups) + 7) / 8 * 8 + (ngroups ? (ngroups + 1) * 8 : 0);
    const AttFn merge = ngroups ? att_shared_merge(D, P, pl.rt) : att_merge_of<ATT_PLAIN>(D, P, pl.rt);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, merge, (const AttParams)p);
    return e == cudaSuccess ? MK_OK : serve_cuda_fail(e, "attention merge launch");
}

static int shared_check(const mk_attend_desc *a, const mk_shared_desc *s) {
    if (!a || !s) return set_error(MK_ERR_INVALID, "null descriptor");
    if (s->groups < 0) return set_error(MK_ERR_INVALID, "negative number of groups");
    if (s->groups > a->batch || (int64_t)s->groups + a->batch > ATT_MAXB)
        return set_error(MK_ERR_UNSUPPORTED, "more groups than sequences, or more than 1024 of both in one call");
    if (a->window || a->sinks) return set_error(MK_ERR_UNSUPPORTED, "shared prefixes with a window");
    return MK_OK;
}

}  // namespace mk

using namespace mk;

extern "C" {

int mk_cache_attend_workspace(const mk_cache_desc *cache, const mk_attend_desc *attend, uint64_t *bytes) {
    AttPlan pl;
    if (!bytes) return set_error(MK_ERR_INVALID, "bytes is null");
    if (int rc = att_plan(cache, attend, 0, pl)) return rc;
    *bytes = pl.bytes();
    return MK_OK;
}

int mk_cache_attend(const mk_cache_desc *cache, int layer, const mk_attend_desc *a, void *workspace,
                    uint64_t workspace_bytes, void *stream) {
    return att_launch(cache, layer, a, nullptr, workspace, workspace_bytes, stream);
}

int mk_cache_attend_shared_workspace(const mk_cache_desc *cache, const mk_attend_desc *attend,
                                     const mk_shared_desc *shared, uint64_t *bytes) {
    AttPlan pl;
    if (!bytes) return set_error(MK_ERR_INVALID, "bytes is null");
    if (int rc = shared_check(attend, shared)) return rc;
    // (of as many groups or fewer: one group's tiles are the tallest)
    if (int rc = att_plan(cache, attend, shared->groups ? 1 : 0, pl)) return rc;
    *bytes = pl.bytes();
    return MK_OK;
}

int mk_cache_attend_shared(const mk_cache_desc *cache, int layer, const mk_attend_desc *a, const mk_shared_desc *shared,
                           void *workspace, uint64_t workspace_bytes, void *stream) {
    if (int rc = shared_check(a, shared)) return rc;
    if (shared->groups && (!shared->first || !shared->shared || (shared->first | shared->shared) % 4))
        return set_error(MK_ERR_INVALID, "groups and shared must be aligned device arrays");
    return att_launch(cache, layer, a, shared, workspace, workspace_bytes, stream);
}

}  // extern "C"
