// pages_api.hip -- C ABI of the pages of a paged key-value cache (declared in
// include/gemv_pages.h): validation and launch.
#include "gemv_pages.h"

#include "attention_host.hpp"
#include "pages_kernels.hpp"

#include <initializer_list>

namespace gpages {
namespace {

using gattn::aligned;
using gattn::launch;

constexpr int kMostSequences = 65536;   // of a release, whose workgroups each sum over those before theirs

int check(const gemv_page_pool* c, Pool* out)
{
    if (c == nullptr || c->pages < 0 || c->page_size < 1 || c->width < 0 || c->batch < 0 || c->table_stride < c->width)
        return GEMV_E_INVAL;
    if (c->count == nullptr || (c->pages > 0 && c->free_pages == nullptr) ||
        (c->batch > 0 && c->width > 0 && c->table == nullptr))
        return GEMV_E_INVAL;
    *out = Pool{c->free_pages, c->count, c->pages, c->page_size, gattn::divider(c->page_size), c->table, c->table_stride,
                c->width, c->batch};
    return GEMV_OK;
}

struct Span {
    const void* at;
    int64_t bytes;
};

// That outputs share no memory with each other or with inputs, which other
// workgroups still read while the first one writes.
bool apart(std::initializer_list<Span> outs, std::initializer_list<Span> ins)
{
    auto meet = [](const Span& a, const Span& b) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(a.at), q = reinterpret_cast<uintptr_t>(b.at);
        return a.bytes > 0 && b.bytes > 0 && p < q + (uintptr_t)b.bytes && q < p + (uintptr_t)a.bytes;
    };
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        for (const Span* other = o + 1; other != outs.end(); ++other)
            if (meet(*o, *other))
                return false;
        for (const Span& in : ins)
            if (meet(*o, in))
                return false;
    }
    return true;
}

// the entries of a table whose rows follow each other; of another, its first row's
Span entries(const gemv_page_pool* c)
{
    const int64_t rows = c->batch == 0 ? 0 : c->table_stride == c->width ? c->batch : 1;
    return Span{c->table, rows * c->width * (int64_t)sizeof(int32_t)};
}

}  // namespace
}  // namespace gpages

extern "C" {

int gemv_reserve_pages(const gemv_page_pool* pool, const int32_t* lens, const int32_t* added, int rows,
                       int32_t* count_out, int32_t* lens_out, int32_t* starts, int32_t* positions, int64_t* slots,
                       hipStream_t stream)
{
    using namespace gpages;
    Reserve a{};
    if (int rc = check(pool, &a.pool); rc != GEMV_OK)
        return rc;
    if (rows < 0 || count_out == nullptr || starts == nullptr ||
        (pool->batch > 0 && (lens == nullptr || added == nullptr || lens_out == nullptr)) ||
        (rows > 0 && (positions == nullptr || slots == nullptr)))
        return GEMV_E_INVAL;
    if (rows > (int)kMost)
        return GEMV_E_UNSUPPORTED;
    const int64_t each = (int64_t)pool->batch * (int64_t)sizeof(int32_t);
    if (!apart({{count_out, 8}, {lens_out, each}, {starts, each + 4}, {positions, 4 * (int64_t)rows}, {slots, 8 * (int64_t)rows}},
               {{pool->count, 4}, {pool->free_pages, 4 * (int64_t)pool->pages}, entries(pool), {lens, each}, {added, each}}))
        return GEMV_E_INVAL;
    a.lens = lens;
    a.added = added;
    a.rows = rows;
    a.count_out = count_out;
    a.lens_out = lens_out;
    a.starts = starts;
    a.positions = positions;
    a.slots = slots;
    void* args[] = {(void*)&a};
    const int64_t grid = ((int64_t)rows + kRows - 1) / kRows;
    return launch(reinterpret_cast<const void*>(&reserve_kernel), grid > 0 ? grid : 1, kThreads, args, stream);
}

size_t gemv_release_pages_workspace(const gemv_page_pool* pool)
{
    using namespace gpages;
    Pool p{};
    return check(pool, &p) == GEMV_OK && p.batch <= kMostSequences ? (size_t)p.batch * sizeof(int32_t) : 0;
}

int gemv_release_pages(const gemv_page_pool* pool, const int32_t* keep, int32_t* count_out, void* workspace,
                       size_t workspace_bytes, hipStream_t stream)
{
    using namespace gpages;
    Release a{};
    if (int rc = check(pool, &a.pool); rc != GEMV_OK)
        return rc;
    if (count_out == nullptr || count_out == pool->count || (pool->batch > 0 && keep == nullptr))
        return GEMV_E_INVAL;
    if (pool->batch > kMostSequences)
        return GEMV_E_UNSUPPORTED;
    const size_t need = gemv_release_pages_workspace(pool);
    if (need > 0 && (workspace == nullptr || workspace_bytes < need || !aligned(workspace, 16)))
        return GEMV_E_INVAL;
    if (!apart({{count_out, 8}, {workspace, (int64_t)need}},
               {{pool->count, 4}, {pool->free_pages, 4 * (int64_t)pool->pages}, entries(pool),
                {keep, (int64_t)pool->batch * (int64_t)sizeof(int32_t)}}))
        return GEMV_E_INVAL;
    a.keep = keep;
    a.count_out = count_out;
    a.given = static_cast<int32_t*>(workspace);
    void* args[] = {(void*)&a};
    if (pool->batch > 0)
        if (int rc = launch(reinterpret_cast<const void*>(&count_kernel), pool->batch, kReleaseThreads, args, stream); rc != GEMV_OK)
            return rc;
    return launch(reinterpret_cast<const void*>(&release_kernel), pool->batch > 0 ? pool->batch : 1, kReleaseThreads, args, stream);
}

}  // extern "C"
