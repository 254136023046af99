// Host accounting of a cache's pages: reference counts, lowest-numbered free
// page first (so that a pool that empties can be compacted cheaply).
#include <new>

#include "planner.h"

struct mk_pages_s {
    std::vector<int32_t> refs;
    int free_pages = 0;
    int lowest = 0;  // no free page lies below
};

using mk::set_error;

// MK_OK if every id is in range and its page in use.
static int each_in_use(const mk_pages_s &p, const int32_t *ids, int n) {
    for (int i = 0; i < n; ++i) {
        if (ids[i] < 0 || ids[i] >= (int)p.refs.size()) return set_error(MK_ERR_INVALID, "page number out of range");
        if (p.refs[ids[i]] <= 0) return set_error(MK_ERR_INVALID, "page " + std::to_string(ids[i]) + " is not in use");
    }
    return MK_OK;
}

extern "C" {

int mk_pages_create(int num_pages, mk_pages_t *out) {
    if (!out) return set_error(MK_ERR_INVALID, "out is null");
    *out = nullptr;
    if (num_pages <= 0) return set_error(MK_ERR_INVALID, "num_pages must be positive");
    try {
        auto *p = new mk_pages_s;
        try {
            p->refs.assign(num_pages, 0);
        } catch (const std::bad_alloc &) {
            delete p;
            throw;
        }
        p->free_pages = num_pages;
        *out = p;
    } catch (const std::bad_alloc &) {
        return set_error(MK_ERR_INVALID, "out of host memory");
    }
    return MK_OK;
}

int mk_pages_alloc(mk_pages_t p, int n, int32_t *ids) {
    if (!p || n < 0 || (n > 0 && !ids)) return set_error(MK_ERR_INVALID, "null argument or negative count");
    if (n > p->free_pages)
        return set_error(MK_ERR_INVALID, "out of pages: " + std::to_string(n) + " wanted, " + std::to_string(p->free_pages) + " free");
    int at = p->lowest;
    for (int i = 0; i < n; ++i, ++at) {
        while (p->refs[at]) ++at;
        p->refs[at] = 1;
        ids[i] = at;
    }
    if (n > 0) p->lowest = at;
    p->free_pages -= n;
    return MK_OK;
}

int mk_pages_share(mk_pages_t p, const int32_t *ids, int n) {
    if (!p || n < 0 || (n > 0 && !ids)) return set_error(MK_ERR_INVALID, "null argument or negative count");
    if (int rc = each_in_use(*p, ids, n)) return rc;
    for (int i = 0; i < n; ++i) {
        if (p->refs[ids[i]] == INT32_MAX) {
            while (i-- > 0) --p->refs[ids[i]];
            return set_error(MK_ERR_INVALID, "too many references to a page");
        }
        ++p->refs[ids[i]];
    }
    return MK_OK;
}

int mk_pages_release(mk_pages_t p, const int32_t *ids, int n) {
    if (!p || n < 0 || (n > 0 && !ids)) return set_error(MK_ERR_INVALID, "null argument or negative count");
    if (int rc = each_in_use(*p, ids, n)) return rc;
    for (int i = 0; i < n; ++i) {
        if (p->refs[ids[i]] == 0) {  // listed more often than referenced
            const int bad = ids[i];
            while (i-- > 0)
                if (p->refs[ids[i]]++ == 0) --p->free_pages;
            return set_error(MK_ERR_INVALID, "page " + std::to_string(bad) + " is released more often than it is held");
        }
        if (--p->refs[ids[i]] == 0) ++p->free_pages;
    }
    for (int i = 0; i < n; ++i)
        if (p->refs[ids[i]] == 0 && ids[i] < p->lowest) p->lowest = ids[i];
    return MK_OK;
}

int mk_pages_compact(mk_pages_t p, int32_t *src, int32_t *dst, int *n) {
    if (!p || !src || !dst || !n) return set_error(MK_ERR_INVALID, "null argument");
    const int used = (int)p->refs.size() - p->free_pages;
    int lo = 0, k = 0;
    for (int hi = (int)p->refs.size() - 1; hi >= used; --hi) {
        if (!p->refs[hi]) continue;
        while (p->refs[lo]) ++lo;
        src[k] = hi;
        dst[k++] = lo;
        p->refs[lo] = p->refs[hi];
        p->refs[hi] = 0;
    }
    p->lowest = used;
    *n = k;
    return MK_OK;
}

int mk_pages_info(mk_pages_t p, int32_t *refs, int *free_pages) {
    if (!p) return set_error(MK_ERR_INVALID, "null page pool");
    if (refs)
        for (size_t i = 0; i < p->refs.size(); ++i) refs[i] = p->refs[i];
    if (free_pages) *free_pages = p->free_pages;
    return MK_OK;
}

void mk_pages_free(mk_pages_t p) { delete p; }

}  // extern "C"
