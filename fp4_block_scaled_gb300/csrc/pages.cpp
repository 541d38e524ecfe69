// pages.cpp -- which page of the key-value cache holds which tokens of which
// sequence (host code, no GPU).
//
// A sequence is a list of page ids and a length; a page counts the sequences
// that hold it.  Forking copies the list and counts every page once more, so
// it moves no data; the first token that a sequence then writes into a page it
// shares gives it a page of its own and one copy to make.  Free pages are a
// bitset searched from a hint below which none is free, so a new page is the
// lowest free one.  Whatever can run out is taken before anything changes, and
// no C++ exception leaves the library.
#include <stdint.h>

#include <new>
#include <vector>

#include "../../include/moe_ffn.h"

struct moe_kv_pages_s {
    int pages, page_size, max_seqs, row;
    std::vector<int32_t> refs;                   // sequences that hold each page
    std::vector<uint64_t> free_bits;
    int free_count;
    size_t hint = 0;                             // no free page in the words before it
    struct Seq {
        bool open = false;
        int len = 0;
        std::vector<int32_t> ids;
    };
    std::vector<Seq> seqs;
    int seq_hint = 0;                            // no closed id before it

    int take()                                   // the lowest free page; there is one
    {
        while (!free_bits[hint]) hint++;
        const int b = __builtin_ctzll(free_bits[hint]);
        free_bits[hint] &= free_bits[hint] - 1;
        free_count--;
        const int p = (int)(hint * 64) + b;
        refs[(size_t)p] = 1;
        return p;
    }
    void drop(int p)
    {
        if (--refs[(size_t)p] > 0) return;
        free_bits[(size_t)p / 64] |= 1ull << (p % 64);
        free_count++;
        if ((size_t)p / 64 < hint) hint = (size_t)p / 64;
    }
    bool is_open(int s) const { return s >= 0 && s < max_seqs && seqs[(size_t)s].open; }
    int closed_id()
    {
        while (seq_hint < max_seqs && seqs[(size_t)seq_hint].open) seq_hint++;
        return seq_hint < max_seqs ? seq_hint : -1;
    }
};

extern "C" {

int moe_kv_pages_create(int num_pages, int page_size, int max_seqs, int max_pages_per_seq, moe_kv_pages_t* out)
{
    if (!out) return MOE_ERR_INVALID_ARG;
    *out = nullptr;
    if (num_pages <= 0 || page_size <= 0 || max_seqs <= 0 || max_pages_per_seq <= 0 ||
        (long long)max_pages_per_seq * page_size > INT32_MAX)
        return MOE_ERR_INVALID_ARG;
    moe_kv_pages_s* m = nullptr;
    try {
        m = new moe_kv_pages_s();
        m->pages = num_pages;
        m->page_size = page_size;
        m->max_seqs = max_seqs;
        m->row = max_pages_per_seq;
        m->refs.assign((size_t)num_pages, 0);
        m->free_bits.assign(((size_t)num_pages + 63) / 64, ~0ull);
        if (num_pages % 64) m->free_bits.back() = (1ull << (num_pages % 64)) - 1;
        m->free_count = num_pages;
        m->seqs.resize((size_t)max_seqs);
    } catch (...) {
        delete m;
        return MOE_ERR_OOM;
    }
    *out = m;
    return MOE_OK;
}

int moe_kv_pages_open(moe_kv_pages_t m, int* seq)
{
    if (!m || !seq) return MOE_ERR_INVALID_ARG;
    const int id = m->closed_id();
    if (id < 0) return MOE_ERR_OOM;
    m->seqs[(size_t)id].open = true;
    m->seqs[(size_t)id].len = 0;
    *seq = id;
    return MOE_OK;
}

int moe_kv_pages_extend(moe_kv_pages_t m, int seq, int tokens, int32_t* copy)
{
    if (!m || !copy || tokens < 0 || !m->is_open(seq)) return MOE_ERR_INVALID_ARG;
    auto& s = m->seqs[(size_t)seq];
    copy[0] = copy[1] = -1;
    if (tokens == 0) return MOE_OK;
    const long long len = (long long)s.len + tokens;
    if (len > (long long)m->row * m->page_size) return MOE_ERR_INVALID_ARG;
    const size_t need = (size_t)((len + m->page_size - 1) / m->page_size);
    const bool inside = s.len % m->page_size != 0;
    const bool split = inside && m->refs[(size_t)s.ids.back()] > 1;
    if (need - s.ids.size() + (split ? 1 : 0) > (size_t)m->free_count) return MOE_ERR_OOM;
    try {
        if (s.ids.capacity() < need) s.ids.reserve(need > 2 * s.ids.capacity() ? need : 2 * s.ids.capacity());
    } catch (...) {
        return MOE_ERR_OOM;
    }
    if (split) {
        copy[0] = s.ids.back();
        m->drop(copy[0]);
        copy[1] = s.ids.back() = m->take();
    }
    while (s.ids.size() < need) s.ids.push_back(m->take());
    s.len = (int)len;
    return MOE_OK;
}

int moe_kv_pages_fork(moe_kv_pages_t m, int parent, int* seq)
{
    if (!m || !seq || !m->is_open(parent)) return MOE_ERR_INVALID_ARG;
    const int id = m->closed_id();
    if (id < 0) return MOE_ERR_OOM;
    auto& p = m->seqs[(size_t)parent];
    auto& s = m->seqs[(size_t)id];
    try {
        s.ids = p.ids;
    } catch (...) {
        s.ids.clear();
        return MOE_ERR_OOM;
    }
    for (int32_t page : s.ids) m->refs[(size_t)page]++;
    s.len = p.len;
    s.open = true;
    *seq = id;
    return MOE_OK;
}

int moe_kv_pages_free(moe_kv_pages_t m, int seq)
{
    if (!m || !m->is_open(seq)) return MOE_ERR_INVALID_ARG;
    auto& s = m->seqs[(size_t)seq];
    for (int32_t page : s.ids) m->drop(page);
    s.ids.clear();
    s.len = 0;
    s.open = false;
    if (seq < m->seq_hint) m->seq_hint = seq;
    return MOE_OK;
}

int moe_kv_pages_compact(moe_kv_pages_t m, int32_t* pairs, int max_pairs, int* n)
{
    if (!m || !n || max_pairs < 0 || (max_pairs > 0 && !pairs)) return MOE_ERR_INVALID_ARG;
    *n = 0;
    const int used = m->pages - m->free_count;
    std::vector<int32_t> to;                     // where the pages from `used` on go
    try {
        to.assign((size_t)(m->pages - used), -1);
    } catch (...) {
        return MOE_ERR_OOM;
    }
    int moved = 0;
    for (int p = used; p < m->pages && moved < max_pairs; p++) {
        if (!m->refs[(size_t)p]) continue;
        const int32_t count = m->refs[(size_t)p];
        const int d = m->take();                 // below `used`: as many are free there as used above
        m->refs[(size_t)d] = count;
        m->refs[(size_t)p] = 0;
        to[(size_t)(p - used)] = d;
        pairs[2 * moved] = p;
        pairs[2 * moved + 1] = d;
        moved++;
    }
    if (moved) {
        for (auto& s : m->seqs)
            for (int32_t& id : s.ids)
                if (id >= used && to[(size_t)(id - used)] >= 0) id = to[(size_t)(id - used)];
        for (int i = 0; i < moved; i++) {        // the places left become free
            const int p = pairs[2 * i];
            m->free_bits[(size_t)p / 64] |= 1ull << (p % 64);
            m->free_count++;
        }
    }
    *n = moved;
    return MOE_OK;
}

int moe_kv_pages_row(moe_kv_pages_t m, int seq, int32_t* row, int entries)
{
    if (!m || !row || !m->is_open(seq)) return MOE_ERR_INVALID_ARG;
    const auto& ids = m->seqs[(size_t)seq].ids;
    if (entries < 0 || ids.size() > (size_t)entries) return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < entries; i++) row[i] = (size_t)i < ids.size() ? ids[(size_t)i] : -1;
    return MOE_OK;
}

int moe_kv_pages_length(moe_kv_pages_t m, int seq)
{
    return m && m->is_open(seq) ? m->seqs[(size_t)seq].len : MOE_ERR_INVALID_ARG;
}

int moe_kv_pages_free_pages(moe_kv_pages_t m) { return m ? m->free_count : MOE_ERR_INVALID_ARG; }

int moe_kv_pages_refs(moe_kv_pages_t m, int page)
{
    return m && page >= 0 && page < m->pages ? m->refs[(size_t)page] : MOE_ERR_INVALID_ARG;
}

void moe_kv_pages_destroy(moe_kv_pages_t m) { delete m; }

}  // extern "C"
