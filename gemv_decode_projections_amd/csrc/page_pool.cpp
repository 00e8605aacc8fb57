// The page pool (include/block.h, blk_pool_*): which pages of a cache are in
// use, and by how many sequences. Host memory only.
#include <stdint.h>

#include <algorithm>
#include <new>
#include <vector>

#include "../../include/block.h"
#include "../../include/proj.h"

// Counts per page, and a bitmap of the free ones: the lowest free page is
// found from the first word that may hold one, so allocation keeps the pages
// in use at the cache's beginning and a compaction moves little.
struct blk_pool {
    std::vector<int32_t> users;
    std::vector<uint64_t> free_bits;
    size_t first_word = 0;             // no free page in the words before
    int n_free = 0;

    explicit blk_pool(int n) : users(n, 0), free_bits((n + 63) / 64, 0), n_free(n)
    {
        for (int p = 0; p < n; ++p)
            free_bits[p / 64] |= (uint64_t)1 << (p % 64);
    }
    bool in_use(int32_t p) const { return p >= 0 && (size_t)p < users.size() && users[p] > 0; }
    bool is_free(int32_t p) const { return free_bits[p / 64] >> (p % 64) & 1; }
    int32_t take()                     // n_free > 0
    {
        while (!free_bits[first_word])
            ++first_word;
        const int32_t p = (int32_t)(first_word * 64) + __builtin_ctzll(free_bits[first_word]);
        free_bits[first_word] &= free_bits[first_word] - 1;
        users[p] = 1;
        --n_free;
        return p;
    }
    // Page p, without users now, is free.
    void give(int32_t p)
    {
        free_bits[p / 64] |= (uint64_t)1 << (p % 64);
        first_word = std::min(first_word, (size_t)p / 64);
        ++n_free;
    }
};

extern "C" {

int blk_pool_create(int n_pages, blk_pool **pool)
{
    if (!pool)
        return PROJ_ERR_NULL;
    *pool = nullptr;
    if (n_pages < 1)
        return PROJ_ERR_ARG;
    try {
        *pool = new blk_pool(n_pages);
    } catch (const std::bad_alloc &) {
        return PROJ_ERR_PAGES;
    }
    return PROJ_OK;
}

void blk_pool_destroy(blk_pool *pool) { delete pool; }

int blk_pool_free_pages(const blk_pool *pool) { return pool ? pool->n_free : PROJ_ERR_NULL; }

int blk_pool_users(const blk_pool *pool, int32_t page)
{
    if (!pool)
        return PROJ_ERR_NULL;
    return page >= 0 && (size_t)page < pool->users.size() ? pool->users[page] : PROJ_ERR_ARG;
}

int blk_pool_alloc(blk_pool *pool, int n, int32_t *pages)
{
    if (!pool || (n > 0 && !pages))
        return PROJ_ERR_NULL;
    if (n < 0)
        return PROJ_ERR_ARG;
    if (n > pool->n_free)
        return PROJ_ERR_PAGES;
    for (int i = 0; i < n; ++i)
        pages[i] = pool->take();
    return PROJ_OK;
}

int blk_pool_share(blk_pool *pool, const int32_t *pages, int n)
{
    if (!pool || (n > 0 && !pages))
        return PROJ_ERR_NULL;
    if (n < 0)
        return PROJ_ERR_ARG;
    for (int i = 0; i < n; ++i) {
        if (pool->in_use(pages[i]) && pool->users[pages[i]] < INT32_MAX) {
            ++pool->users[pages[i]];
            continue;
        }
        while (i-- > 0)
            --pool->users[pages[i]];
        return PROJ_ERR_ARG;
    }
    return PROJ_OK;
}

int blk_pool_release(blk_pool *pool, const int32_t *pages, int n)
{
    if (!pool || (n > 0 && !pages))
        return PROJ_ERR_NULL;
    if (n < 0)
        return PROJ_ERR_ARG;
    for (int i = 0; i < n; ++i) {
        if (pool->in_use(pages[i])) {
            --pool->users[pages[i]];
            continue;
        }
        while (i-- > 0)
            ++pool->users[pages[i]];
        return PROJ_ERR_ARG;
    }
    for (int i = 0; i < n; ++i)
        if (!pool->users[pages[i]] && !pool->is_free(pages[i]))
            pool->give(pages[i]);
    return PROJ_OK;
}

int blk_pool_compact(blk_pool *pool, int max_moves, int32_t *src, int32_t *dst)
{
    if (!pool || (max_moves > 0 && (!src || !dst)))
        return PROJ_ERR_NULL;
    if (max_moves < 0)
        return PROJ_ERR_ARG;
    int moves = 0;
    int32_t high = (int32_t)pool->users.size() - 1;
    while (moves < max_moves && pool->n_free) {
        while (high >= 0 && !pool->users[high])
            --high;
        while (pool->first_word < pool->free_bits.size() && !pool->free_bits[pool->first_word])
            ++pool->first_word;
        const int32_t low = (int32_t)(pool->first_word * 64) + __builtin_ctzll(pool->free_bits[pool->first_word]);
        if (high < low)
            break;
        src[moves] = high;
        dst[moves++] = low;
        const int32_t users = pool->users[high];
        pool->take();                  // low
        pool->users[low] = users;
        pool->users[high] = 0;
        pool->give(high);              // above every page still in use: no later move's target
        --high;
    }
    return moves;
}

}  // extern "C"
