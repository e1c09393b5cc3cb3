// rotate_api.hip -- C ABI of the norms and the rotation of queries and keys
// (declared in include/gemv_rotate.h): validation, geometry and launch.
#include "gemv_rotate.h"

#include "device_info.hpp"
#include "rotate_kernels.hpp"

#include <numeric>

namespace grot {
namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool is_type(int t) { return t == GEMV_F32 || t == GEMV_F16 || t == GEMV_BF16; }

int check_how(const gemv_rotation* how, int dtype, int rows)
{
    if (how == nullptr || rows < 0 || !is_type(dtype) || how->head_dim < 1 || how->rotated < 0 ||
        how->rotated > how->head_dim || how->rotated % 2 != 0 || (how->norm != 0 && !is_type(how->weight_dtype)))
        return GEMV_E_INVAL;
    return how->head_dim > kMaxDim ? GEMV_E_UNSUPPORTED : GEMV_OK;
}

int check_heads(const gemv_heads* h, int dim, int rows, bool own_out)
{
    const int64_t width = h->heads < 0 ? -1 : (int64_t)h->heads * dim;
    if (width < 0 || h->stride < width || (own_out && h->out_stride < width))
        return GEMV_E_INVAL;
    if (rows > 0 && width > 0 && (h->x == nullptr || (own_out && h->out == nullptr)))
        return GEMV_E_INVAL;
    return GEMV_OK;
}

int bytes_of(int type) { return type == GEMV_F32 ? 4 : 2; }

// Rows of `width` bytes, `step` apart.
struct Rows {
    uintptr_t at, width, step;
};

Rows inputs_of(const gemv_heads* h, int dim, int type)
{
    const uintptr_t size = bytes_of(type);
    return Rows{reinterpret_cast<uintptr_t>(h->x), (uintptr_t)h->heads * dim * size, (uintptr_t)h->stride * size};
}

Rows outputs_of(const gemv_heads* h, int dim, int type)
{
    const uintptr_t size = bytes_of(type);
    return Rows{reinterpret_cast<uintptr_t>(h->out), (uintptr_t)h->heads * dim * size, (uintptr_t)h->out_stride * size};
}

// Whether some row of one shares a byte with some row of the other; parts of a
// product's rows, whose rows take turns, do not.
bool meet(Rows a, Rows b, int rows)
{
    if (a.width == 0 || b.width == 0)
        return false;
    if (b.at < a.at) {
        const Rows c = a;
        a = b;
        b = c;
    }
    const uintptr_t n = (uintptr_t)rows;
    if (b.at >= a.at + (n - 1) * a.step + a.width)
        return false;
    if (a.step == b.step) {
        const uintptr_t turns = (b.at - a.at) / a.step, into = (b.at - a.at) % a.step;   // a step is a row at least
        return (turns < n && into < a.width) || (turns + 1 < n && a.step - into < b.width);
    }
    const uintptr_t period = a.step / std::gcd(a.step, b.step);   // rows of b until they lie to a's as before
    for (uintptr_t j = 0; j < n && j < period; ++j) {
        const uintptr_t from = b.at + j * b.step, i = (from - a.at) / a.step, into = (from - a.at) % a.step;
        if (i >= n)
            break;
        if (into < a.width || (i + 1 < n && a.step - into < b.width))
            return true;
    }
    return false;
}

// Results in the place of their own inputs, or apart from all inputs and each other:
// laid over them in another way they would meet elements that are still to be read.
bool placed(const gemv_heads* const* of, int n, int outs, int dim, int in, int out, int rows)
{
    for (int i = 0; i < outs; ++i) {
        const Rows o = outputs_of(of[i], dim, out);
        for (int j = 0; j < n; ++j) {
            const Rows x = inputs_of(of[j], dim, in);
            const bool own = i == j && o.at == x.at && in == out && (o.step == x.step || rows == 1);
            if (!own && meet(o, x, rows))
                return false;
            if (j < outs && j != i && meet(o, outputs_of(of[j], dim, out), rows))
                return false;
        }
    }
    return true;
}

// 16 bytes of every row, head and piece
bool wide(const gemv_heads* h, bool own_out)
{
    return aligned(h->x, 16) && h->stride % 8 == 0 && aligned(h->weight, 16) &&
           (!own_out || (aligned(h->out, 16) && h->out_stride % 8 == 0));
}

// a row's steps are counted in int, and no head is smaller than a step
bool countable(const gemv_heads* const* of, int n)
{
    int64_t heads = 0;
    for (int i = 0; i < n; ++i)
        heads += of[i]->heads;
    return heads <= gemv_device::kMaxWorkItems;
}

constexpr int kElements = -1;   // in the place of a pairing: element by element

template <int IN, int OUT>
const void* kernel_for(int pairing)
{
    return pairing == kHalves       ? reinterpret_cast<const void*>(&rotate_kernel<IN, OUT, kHalves>)
           : pairing == kNeighbours ? reinterpret_cast<const void*>(&rotate_kernel<IN, OUT, kNeighbours>)
           : pairing == kLoose      ? reinterpret_cast<const void*>(&rotate_kernel<IN, OUT, kLoose>)
                                    : reinterpret_cast<const void*>(&rotate_elementwise<IN, OUT>);
}

template <int IN>
const void* kernel_for(int out, int pairing)
{
    return out == GEMV_F32 ? kernel_for<IN, kF32>(pairing) : out == GEMV_F16 ? kernel_for<IN, kF16>(pairing)
                                                                             : kernel_for<IN, kBF16>(pairing);
}

int run(Rotate& a, bool vector, int in, int out, hipStream_t stream)
{
    gemv_device::Device dev{};
    if (int rc = gemv_device::current(&dev); rc != GEMV_OK)
        return rc;
    int per = 1, pairing = kElements;
    if (vector) {
        const int half = a.rotated / 2;
        pairing = a.interleaved ? kNeighbours : half % 8 == 0 ? kHalves : kLoose;
        a.units = pairing == kHalves ? half / 8 + ((a.dim - a.rotated) / 8 + 1) / 2 : (a.dim / 8 + 1) / 2;
        a.lanes = 1;
        while (a.lanes < a.units)
            a.lanes *= 2;
        per = 64 / a.lanes;
    }
    for (Heads& h : a.of)
        h.turns = (h.heads + per - 1) / per;
    a.turns = a.of[0].turns + a.of[1].turns + a.of[2].turns;
    if (a.turns == 0 || a.rows == 0)
        return GEMV_OK;
    // a row's steps are shared out among waves only until there are about twelve a CU:
    // its angles are taken by each of them (8191 rows of 32 + 8 + 8 heads of 128, six
    // steps: 46.9 us by one wave, 55.2 by three; 1000 rows: 14.0 and 9.0); element by
    // element the waves wait more
    const int64_t full = (int64_t)dev.cus * (vector ? 12 : 64), share = (full + a.rows / 2) / a.rows;
    const int spans_of = (int)(share < 1 ? 1 : share < a.turns ? share : a.turns);
    a.span = (a.turns + spans_of - 1) / spans_of;
    const int64_t waves = (int64_t)a.rows * ((a.turns + a.span - 1) / a.span);
    const void* fn = in == GEMV_F32   ? kernel_for<kF32>(out, pairing)
                     : in == GEMV_F16 ? kernel_for<kF16>(out, pairing) : kernel_for<kBF16>(out, pairing);
    void* args[] = {(void*)&a};
    const int grid = gemv_device::capped_grid((waves + kWaves - 1) / kWaves, kWaves * 64);
    return hipLaunchKernel(fn, dim3((unsigned)grid), dim3(kWaves * 64), args, 0, stream) == hipSuccess ? GEMV_OK : GEMV_E_LAUNCH;
}

Heads heads_of(const gemv_heads* h, bool norm)
{
    return Heads{h->x, h->stride, h->heads, norm ? h->weight : nullptr, h->out, h->out_stride, 0};
}

Rotate rotation_of(const gemv_rotation* how, const int32_t* positions, int rows)
{
    Rotate a{};
    a.positions = positions;
    a.rows = rows;
    a.dim = how->head_dim;
    a.rotated = how->rotated;
    a.per_element = 1.0f / (float)how->head_dim;
    a.interleaved = how->interleaved != 0;
    a.norm = how->norm != 0;
    a.eps = how->eps;
    a.freqs = how->freqs;
    a.weight_dtype = how->weight_dtype;
    return a;
}

bool pieces(const gemv_rotation* how) { return how->head_dim % 8 == 0; }

}  // namespace
}  // namespace grot

extern "C" {

int gemv_norm_rotate(const gemv_rotation* how, const gemv_heads* q, const gemv_heads* k, int dtype, int out_dtype,
                     const int32_t* positions, int rows, hipStream_t stream)
{
    using namespace grot;
    if (int rc = check_how(how, dtype, rows); rc != GEMV_OK)
        return rc;
    if (q == nullptr || !is_type(out_dtype))
        return GEMV_E_INVAL;
    bool vector = pieces(how) && wide(q, true);
    if (int rc = check_heads(q, how->head_dim, rows, true); rc != GEMV_OK)
        return rc;
    if (k != nullptr) {
        if (int rc = check_heads(k, how->head_dim, rows, true); rc != GEMV_OK)
            return rc;
        vector = vector && wide(k, true);
    }
    if (rows == 0)
        return GEMV_OK;
    if (positions == nullptr || (how->rotated > 0 && how->freqs == nullptr))
        return GEMV_E_INVAL;
    const gemv_heads* const both[2] = {q, k};
    const int given = k != nullptr ? 2 : 1;
    if (!placed(both, given, given, how->head_dim, dtype, out_dtype, rows))
        return GEMV_E_INVAL;
    if (!countable(both, given))
        return GEMV_E_UNSUPPORTED;
    Rotate a = rotation_of(how, positions, rows);
    a.of[kQuery] = heads_of(q, a.norm);
    if (k != nullptr)
        a.of[kKey] = heads_of(k, a.norm);
    return run(a, vector, dtype, out_dtype, stream);
}

int gemv_norm_rotate_append(const gemv_rotation* how, const gemv_heads* q, const gemv_heads* k, const gemv_heads* v,
                            int dtype, const int32_t* positions, int rows, const gemv_kv_cache* cache,
                            const int64_t* slots, hipStream_t stream)
{
    using namespace grot;
    if (int rc = check_how(how, dtype, rows); rc != GEMV_OK)
        return rc;
    if (q == nullptr || k == nullptr || v == nullptr || cache == nullptr)
        return GEMV_E_INVAL;
    if (cache->pages < 0 || cache->page_size < 1 || cache->heads < 1 || cache->head_dim != how->head_dim ||
        (cache->dtype != GEMV_F16 && cache->dtype != GEMV_BF16) || k->heads != cache->heads || v->heads != cache->heads ||
        cache->stride_page < cache->head_dim || cache->stride_slot < cache->head_dim || cache->stride_head < cache->head_dim)
        return GEMV_E_INVAL;
    for (const gemv_heads* h : {q, k, v})
        if (int rc = check_heads(h, how->head_dim, rows, h == q); rc != GEMV_OK)
            return rc;
    if (cache->head_dim % 8 != 0 || cache->stride_page % 8 != 0 || cache->stride_slot % 8 != 0 || cache->stride_head % 8 != 0 ||
        !aligned(cache->k, 16) || !aligned(cache->v, 16))
        return GEMV_E_UNSUPPORTED;
    if (rows == 0)
        return GEMV_OK;
    const gemv_heads* const all[3] = {q, k, v};
    if (!placed(all, 3, 1, how->head_dim, dtype, cache->dtype, rows))
        return GEMV_E_INVAL;
    if (!countable(all, 3))
        return GEMV_E_UNSUPPORTED;
    if (positions == nullptr || slots == nullptr || (how->rotated > 0 && how->freqs == nullptr) ||
        (cache->pages > 0 && (cache->k == nullptr || cache->v == nullptr)))
        return GEMV_E_INVAL;
    Rotate a = rotation_of(how, positions, rows);
    a.of[kQuery] = heads_of(q, a.norm);
    a.of[kKey] = heads_of(k, a.norm);
    a.of[kValue] = heads_of(v, false);
    a.of[kKey].out = cache->k;
    a.of[kValue].out = cache->v;
    a.slots = slots;
    a.pages = cache->pages;
    a.stride_page = cache->stride_page;
    a.stride_slot = cache->stride_slot;
    a.stride_head = cache->stride_head;
    a.page_size = cache->page_size;
    gemv_heads plain = *v;
    plain.weight = nullptr;
    return run(a, pieces(how) && wide(q, true) && wide(k, false) && wide(&plain, false), dtype, cache->dtype, stream);
}

}  // extern "C"
