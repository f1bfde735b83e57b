// The pager of the paged private caches: which pages each sequence owns.
// Host only. Pages are reference counted and searched from a hint below which
// none is free, so that the lowest free page is always the one taken (a cache that shrinks keeps its owned pages low, and the same calls
// always give the same pages).
#include <limits.h>
#include <stdint.h>

#include <algorithm>
#include <new>
#include <vector>

#include "kvpool.h"

struct kvpool_pager {
    struct Seq {
        bool live = false;
        int len = 0;
        std::vector<int32_t> table;
    };
    int pages = 0, page_tokens = 0, nfree = 0;
    int low = 0;                 // no page below is free
    std::vector<int32_t> owners; // per page; 0: free
    std::vector<Seq> seqs;

    bool has(int s) const { return s >= 0 && s < (int)seqs.size() && seqs[s].live; }
    int take() {  // the lowest free page (nfree > 0)
        while (owners[low] != 0) ++low;
        owners[low] = 1;
        --nfree;
        return low++;
    }
    void let_go(int page) {
        if (--owners[page] == 0) {
            ++nfree;
            low = std::min(low, page);
        }
    }
    int pages_of(long long tokens) const { return (int)((tokens + page_tokens - 1) / page_tokens); }
    int slot() {  // the lowest unused sequence number
        for (size_t i = 0; i < seqs.size(); ++i)
            if (!seqs[i].live) return (int)i;
        if (seqs.size() >= (size_t)INT_MAX) throw std::bad_alloc();
        seqs.emplace_back();
        return (int)seqs.size() - 1;
    }
};

namespace {

// no C++ exception leaves a C entry
template <class F>
int guarded(F f) {
    try {
        return f();
    } catch (...) {
        return KVPOOL_ERR_OOM;
    }
}

}  // namespace

extern "C" {

int kvpool_pager_create(kvpool_pager_t** out, int pages, int page_tokens) {
    if (!out) return KVPOOL_ERR_INVALID_ARG;
    *out = nullptr;
    if (pages < 1 || (page_tokens != 16 && page_tokens != 32 && page_tokens != 64 && page_tokens != 128))
        return KVPOOL_ERR_INVALID_ARG;
    kvpool_pager* p = new (std::nothrow) kvpool_pager;
    if (!p) return KVPOOL_ERR_OOM;
    const int rc = guarded([&] {
        p->owners.assign(pages, 0);
        return KVPOOL_OK;
    });
    if (rc != KVPOOL_OK) {
        delete p;
        return rc;
    }
    p->pages = p->nfree = pages;
    p->page_tokens = page_tokens;
    *out = p;
    return KVPOOL_OK;
}

void kvpool_pager_destroy(kvpool_pager_t* p) { delete p; }

int kvpool_pager_new(kvpool_pager_t* p) {
    if (!p) return KVPOOL_ERR_INVALID_ARG;
    return guarded([&] {
        const int s = p->slot();
        p->seqs[s].live = true;
        p->seqs[s].len = 0;
        p->seqs[s].table.clear();
        return s;
    });
}

int kvpool_pager_extend(kvpool_pager_t* p, int seq, int n, int32_t copy[2]) {
    if (!p || !p->has(seq) || n < 0 || !copy) return KVPOOL_ERR_INVALID_ARG;
    kvpool_pager::Seq& s = p->seqs[seq];
    if (n > INT_MAX - s.len) return KVPOOL_ERR_INVALID_ARG;
    if (n == 0) return 0;
    return guarded([&] {
        const bool own = s.len % p->page_tokens != 0 && p->owners[s.table.back()] > 1;
        const int want = p->pages_of((long long)s.len + n);
        const int fresh = want - (int)s.table.size() + (own ? 1 : 0);
        if (fresh > p->nfree) return (int)KVPOOL_ERR_OOM;
        // may throw, before anything has changed; doubled, so that growing token by token stays cheap
        if (want > (int)s.table.capacity()) s.table.reserve(std::max<size_t>(want, 2 * s.table.capacity()));
        if (own) {
            copy[0] = s.table.back();
            copy[1] = p->take();
            p->let_go(copy[0]);
            s.table.back() = copy[1];
        }
        while ((int)s.table.size() < want) s.table.push_back(p->take());
        s.len += n;
        return own ? 1 : 0;
    });
}

int kvpool_pager_truncate(kvpool_pager_t* p, int seq, int len) {
    if (!p || !p->has(seq) || len < 0 || len > p->seqs[seq].len) return KVPOOL_ERR_INVALID_ARG;
    kvpool_pager::Seq& s = p->seqs[seq];
    const int keep = p->pages_of(len);
    while ((int)s.table.size() > keep) {
        p->let_go(s.table.back());
        s.table.pop_back();
    }
    s.len = len;
    return KVPOOL_OK;
}

int kvpool_pager_fork(kvpool_pager_t* p, int seq) {
    if (!p || !p->has(seq)) return KVPOOL_ERR_INVALID_ARG;
    return guarded([&] {
        std::vector<int32_t> table = p->seqs[seq].table;
        const int t = p->slot();  // may move the sequences
        p->seqs[t].table.swap(table);
        p->seqs[t].len = p->seqs[seq].len;
        p->seqs[t].live = true;
        for (int32_t page : p->seqs[t].table) ++p->owners[page];
        return t;
    });
}

int kvpool_pager_free(kvpool_pager_t* p, int seq) {
    const int rc = kvpool_pager_truncate(p, seq, 0);
    if (rc == KVPOOL_OK) p->seqs[seq].live = false;
    return rc;
}

int kvpool_pager_compact(kvpool_pager_t* p, int32_t* src, int32_t* dst, int max_pairs) {
    if (!p || max_pairs < 0 || (max_pairs > 0 && (!src || !dst))) return KVPOOL_ERR_INVALID_ARG;
    return guarded([&] {
        std::vector<int32_t> to(p->pages);  // where each page goes
        for (int i = 0; i < p->pages; ++i) to[i] = i;
        // the highest owned pages into the lowest free ones: sources lie at or
        // above the number of owned pages, destinations below it
        int n = 0, lo = 0, hi = p->pages - 1;
        while (n < max_pairs) {
            while (lo < p->pages && p->owners[lo] != 0) ++lo;
            while (hi >= 0 && p->owners[hi] == 0) --hi;
            if (lo >= hi) break;
            src[n] = hi;
            dst[n] = lo;
            to[hi] = lo;
            p->owners[lo] = p->owners[hi];
            p->owners[hi] = 0;
            ++n;
        }
        for (auto& s : p->seqs)
            for (int32_t& page : s.table) page = to[page];
        p->low = 0;
        return n;
    });
}

int kvpool_pager_len(const kvpool_pager_t* p, int seq) {
    if (!p || !p->has(seq)) return KVPOOL_ERR_INVALID_ARG;
    return p->seqs[seq].len;
}

int kvpool_pager_table(const kvpool_pager_t* p, int seq, int32_t* table, int max) {
    if (!p || !p->has(seq) || max < 0 || (max > 0 && !table)) return KVPOOL_ERR_INVALID_ARG;
    const auto& t = p->seqs[seq].table;
    for (int i = 0; i < max && i < (int)t.size(); ++i) table[i] = t[i];
    return (int)t.size();
}

int kvpool_pager_free_pages(const kvpool_pager_t* p) { return p ? p->nfree : KVPOOL_ERR_INVALID_ARG; }

int kvpool_pager_owners(const kvpool_pager_t* p, int page) {
    if (!p || page < 0 || page >= p->pages) return KVPOOL_ERR_INVALID_ARG;
    return p->owners[page];
}

}  // extern "C"
