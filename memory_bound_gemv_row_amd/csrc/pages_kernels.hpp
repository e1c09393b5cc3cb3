// pages_kernels.hpp -- gfx950 (CDNA4) device code for the pages of a paged
// key-value cache: taken for new tokens, with the tokens' slots, and given back.
//
// A few bytes a token, so a launch's latency bounds a decode step, and the
// stores of rows a prompt.
#pragma once

#include "paged.hpp"

namespace gpages {

using gattn::Divider;

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr int kRows = 2048;              // of a workgroup
constexpr unsigned kMost = 1u << 30;     // sums of rows stop here: two of them still fit 32 bits

struct Pool {
    int32_t* free_pages;
    const int32_t* count;
    int pages, page_size;
    Divider page_of;
    int32_t* table;
    int64_t table_stride;
    int width, batch;
};

struct Reserve {
    Pool pool;
    const int32_t* lens;
    const int32_t* added;
    int rows;
    int32_t* count_out;
    int32_t* lens_out;
    int32_t* starts;
    int32_t* positions;
    int64_t* slots;
};

__device__ __forceinline__ unsigned add_rows(unsigned a, unsigned b)
{
    const unsigned s = a + b;
    return s < kMost ? s : kMost;
}

// The sum over the threads before this one, and over all; `waves` holds a value a wave.
__device__ __forceinline__ unsigned scan_threads(unsigned v, unsigned* waves, unsigned* total)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const unsigned u = __shfl_up(v, d);
        v = lane >= d ? add_rows(v, u) : v;
    }
    if (lane == 63)
        waves[wave] = v;
    __syncthreads();
    unsigned before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
        before = w < wave ? add_rows(before, waves[w]) : before;
        all = add_rows(all, waves[w]);
    }
    *total = all;
    __syncthreads();
    v = __shfl_up(v, 1);
    return lane > 0 ? add_rows(v, before) : before;
}

__device__ __forceinline__ int pages_for(int64_t tokens, const Divider& by, int page_size)
{
    const int whole = by.by((int)tokens);
    return whole + ((int64_t)whole * page_size < tokens);
}

// A workgroup for 2048 rows.  Each goes through the sequences 512 at a time:
// sums of their new tokens place them among the rows, sums of the pages that
// they need among those of the stack, and the rows that are its own find their
// sequence in LDS.  So one launch does without an order between workgroups:
// the first writes what there is one of a sequence, and the row of a page's
// first token the page's entry, which no other row of the call looks up.  Bound
// by the chain of its loads and sums: 64 sequences of one new token 3.9 us, 24 of
// up to 8191 7 us, 1024 of 190 10.
__global__ void __launch_bounds__(kThreads)
reserve_kernel(Reserve a)
{
    __shared__ unsigned waves[kWaves];
    __shared__ unsigned first[kThreads];       // row
    __shared__ int length[kThreads], got[kThreads], held[kThreads], taken[kThreads];
    const Pool& p = a.pool;
    const int have0 = p.count[0], have = have0 < 0 ? 0 : (have0 < p.pages ? have0 : p.pages);
    const unsigned begin = blockIdx.x * (unsigned)kRows;
    const unsigned end = begin + kRows < (unsigned)a.rows ? begin + kRows : (unsigned)a.rows;
    unsigned row0 = 0, page0 = 0;              // rows and pages of the sequences before this round's
    for (int b0 = 0; b0 < p.batch; b0 += kThreads) {
        const int b = b0 + (int)threadIdx.x;
        int len = 0, add = 0;
        if (b < p.batch) {
            len = a.lens[b] > 0 ? a.lens[b] : 0;
            add = a.added[b] > 0 ? a.added[b] : 0;
        }
        unsigned rows_all, pages_all;
        const unsigned n = (unsigned)add < kMost ? (unsigned)add : kMost;
        unsigned from = add_rows(row0, scan_threads(n, waves, &rows_all)), last = add_rows(from, n);
        from = from < (unsigned)a.rows ? from : (unsigned)a.rows;
        last = last < (unsigned)a.rows ? last : (unsigned)a.rows;
        int mine = (int)(last - from);
        mine = mine < 0x7FFFFFFF - len ? mine : 0x7FFFFFFF - len;
        const int before = pages_for(len, p.page_of, p.page_size);
        int after = pages_for((int64_t)len + mine, p.page_of, p.page_size);
        after = after < p.width ? after : p.width;
        const unsigned need = after > before ? (unsigned)(after - before) : 0u;
        const unsigned ahead = scan_threads(need, waves, &pages_all);
        first[threadIdx.x] = from;
        length[threadIdx.x] = len;
        got[threadIdx.x] = mine;
        held[threadIdx.x] = before;
        taken[threadIdx.x] = (int)(page0 + ahead);
        if (blockIdx.x == 0 && b < p.batch) {
            a.starts[b] = (int)from;
            a.lens_out[b] = len + mine;
        }
        __syncthreads();
        const int count = p.batch - b0 < kThreads ? p.batch - b0 : kThreads;
        const unsigned next0 = add_rows(row0, rows_all), stop = next0 < end ? next0 : end;
        for (unsigned row = (row0 > begin ? row0 : begin) + threadIdx.x; row < stop; row += kThreads) {
            int low = 0, high = count;         // the last sequence that starts at or before the row
            while (high - low > 1) {
                const int mid = (low + high) >> 1;
                if (first[mid] <= row)
                    low = mid;
                else
                    high = mid;
            }
            const int i = (int)(row - first[low]);
            int64_t slot = -1;
            int position = 0x7FFFFFFF;
            if (i < got[low]) {
                position = length[low] + i;
                const int index = p.page_of.by(position), at = position - index * p.page_size;
                if (index < p.width) {
                    int32_t* const entry = p.table + (b0 + low) * p.table_stride + index;
                    int page;
                    if (index < held[low]) {
                        page = *entry;
                    } else {
                        const int nth = taken[low] + index - held[low];
                        page = nth < have ? p.free_pages[have - 1 - nth] : -1;
                        page = (unsigned)page < (unsigned)p.pages ? page : -1;
                        if (at == 0)
                            *entry = page;
                    }
                    if ((unsigned)page < (unsigned)p.pages)
                        slot = (int64_t)page * p.page_size + at;
                }
            }
            a.positions[row] = position;
            a.slots[row] = slot;
        }
        row0 = next0;
        page0 += pages_all;
        if (blockIdx.x != 0 && row0 >= end)
            return;
        __syncthreads();                       // the next round writes what this one's rows read
    }
    for (unsigned row = (row0 > begin ? row0 : begin) + threadIdx.x; row < end; row += kThreads) {
        a.positions[row] = 0;
        a.slots[row] = -1;
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.starts[p.batch] = (int)(row0 < (unsigned)a.rows ? row0 : (unsigned)a.rows);
        a.count_out[0] = have > (int)page0 ? have - (int)page0 : 0;
        a.count_out[1] = (int)page0 > have ? (int)page0 - have : 0;
    }
}

struct Release {
    Pool pool;
    const int32_t* keep;
    int32_t* count_out;
    int32_t* given;          // [batch]: pages that a sequence gives back
};

constexpr int kReleaseThreads = 256;

__device__ __forceinline__ int first_given(const Release& a, int b)
{
    const int keep = a.keep[b] > 0 ? a.keep[b] : 0;
    return pages_for(keep, a.pool.page_of, a.pool.page_size);
}

__device__ __forceinline__ int64_t sum_threads(int64_t v, int64_t* waves)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0)
        waves[threadIdx.x >> 6] = v;
    __syncthreads();
    v = waves[0] + waves[1] + waves[2] + waves[3];
    __syncthreads();
    return v;
}

// A workgroup per sequence: how many pages it gives back.  (With the launch that
// puts them back 4.5 us for 64 sequences of 4000 tokens, 24 for four of 131072,
// whose 8192 entries one workgroup walks.)
__global__ void __launch_bounds__(kReleaseThreads)
count_kernel(Release a)
{
    __shared__ int64_t waves[kReleaseThreads / 64];
    const int b = blockIdx.x;
    const int32_t* row = a.pool.table + b * a.pool.table_stride;
    int64_t n = 0;
    for (int64_t i = (int64_t)first_given(a, b) + threadIdx.x; i < a.pool.width; i += kReleaseThreads)
        n += (unsigned)row[i] < (unsigned)a.pool.pages;
    n = sum_threads(n, waves);
    if (threadIdx.x == 0)
        a.given[b] = (int)n;
}

// And puts them behind those of the sequences before it.
__global__ void __launch_bounds__(kReleaseThreads)
release_kernel(Release a)
{
    __shared__ int64_t waves[kReleaseThreads / 64];
    const Pool& p = a.pool;
    const int have0 = p.count[0], have = have0 < 0 ? 0 : (have0 < p.pages ? have0 : p.pages);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (p.batch == 0) {
        if (threadIdx.x == 0) {
            a.count_out[0] = have;
            a.count_out[1] = 0;
        }
        return;
    }
    const int b = blockIdx.x;
    int64_t before = 0;
    for (int i = threadIdx.x; i < b; i += kReleaseThreads)
        before += a.given[i];
    int64_t at = have + sum_threads(before, waves);
    int32_t* row = p.table + b * p.table_stride;
    for (int64_t base = first_given(a, b); base < p.width; base += kReleaseThreads) {
        const int64_t i = base + threadIdx.x;
        const int page = i < p.width ? row[i] : -1;
        const bool is = (unsigned)page < (unsigned)p.pages;
        const uint64_t mask = __ballot(is);
        if (lane == 0)
            waves[wave] = __popcll(mask);
        __syncthreads();
        int64_t to = at + __popcll(mask & ((1ull << lane) - 1));
        for (int w = 0; w < wave; ++w)
            to += waves[w];
        if (is && to < p.pages)
            p.free_pages[to] = page;
        if (i < p.width)
            row[i] = -1;
        at += waves[0] + waves[1] + waves[2] + waves[3];
        __syncthreads();
    }
    if (b == p.batch - 1 && threadIdx.x == 0) {
        a.count_out[0] = (int)(at < p.pages ? at : p.pages);
        a.count_out[1] = 0;
    }
}

}  // namespace gpages
