// Host-side self-test of the entry points for prompts, prefixes, rotation and pages
// (test infrastructure), built with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/sanitize/serving_build.py and run by tests/test_sanitize_serving_cpu.py.  It
// needs no GPU and no HIP runtime: the few runtime functions that the host code calls
// are defined here, and a launch is kept to be looked at.
//
// Over seeded batches it follows every workgroup of a launch to its key-value head, sequence,
// row tile and part of the keys, by the code that the kernels use where that is not
// for a wave's lanes, and checks that each is taken once, that the parts hold every
// key that a row sees, and that what the workgroups write fits the workspace.
#include "prompt_api.hip"
#include "rotate_api.hip"
#include "pages_api.hip"

#include <stdio.h>
#include <string.h>

#include <map>
#include <tuple>
#include <vector>

// ---------------------------------------------------------------- the runtime
struct Launch {
    const void* fn;
    unsigned grid, block;
    std::vector<unsigned char> first, second;   // the first arguments, copied
    int blocks, count;                          // of a prefix launch
};
static std::vector<Launch> launches;
static size_t sizes[2];   // of the first arguments of the launches to come
static int cus = 256;

extern "C" {
hipError_t hipGetDevice(int* d)
{
    *d = cus == 256 ? 0 : 1;
    return hipSuccess;
}
hipError_t hipDeviceGetAttribute(int* v, hipDeviceAttribute_t what, int)
{
    *v = what == hipDeviceAttributeMultiprocessorCount ? cus : 160 * 1024;
    return hipSuccess;
}
hipError_t hipLaunchKernel(const void* fn, dim3 grid, dim3 block, void** args, size_t, hipStream_t)
{
    Launch l{fn, grid.x, block.x, {}, {}, 0, 0};
    const unsigned char* p = static_cast<const unsigned char*>(args[0]);
    if (launches.empty() && sizes[0] > 0)
        l.first.assign(p, p + sizes[0]);
    if (launches.empty() && sizes[1] > 0) {
        p = static_cast<const unsigned char*>(args[1]);
        l.second.assign(p, p + sizes[1]);
        l.blocks = *static_cast<int*>(args[2]);
        l.count = *static_cast<int*>(args[3]);
    }
    launches.push_back(l);
    return hipSuccess;
}
hipError_t __hipPushCallConfiguration(dim3, dim3, size_t, hipStream_t) { return hipSuccess; }
hipError_t __hipPopCallConfiguration(dim3*, dim3*, size_t*, hipStream_t*) { return hipSuccess; }
void** __hipRegisterFatBinary(const void*)
{
    static void* none;
    return &none;
}
void __hipUnregisterFatBinary(void**) {}
void __hipRegisterFunction(void**, const void*, char*, const char*, unsigned, void*, void*, void*, void*, int*) {}
void __hipRegisterVar(void**, void*, char*, const char*, int, size_t, int, int) {}
}

// ---------------------------------------------------------------- the checks
static int failures = 0;
#define CHECK(c)                                                                                  \
    do {                                                                                          \
        if (!(c) && ++failures < 20)                                                              \
            fprintf(stderr, "check failed at line %d in trial %ld: %s\n", __LINE__, trial, #c);   \
    } while (0)
static long trial = 0;

static uint64_t state = 2027;
static unsigned next()
{
    state = state * 6364136223846793005ull + 1442695040888963407ull;
    return (unsigned)(state >> 33);
}
static int below(int n) { return n > 0 ? (int)(next() % (unsigned)n) : 0; }
template <class T>
static T pick(std::initializer_list<T> of)
{
    return of.begin()[below((int)of.size())];
}

using namespace gattn;

struct Batch {
    std::vector<int32_t> lens, starts;
    int rows, max_new;
};

static int start_of(const Batch& s, int b) { return s.starts[b] < s.rows ? s.starts[b] : s.rows; }

// share_at, a sequence after the other
struct Part {
    int b, part, parts, chunk;
};
static Part part_at(const Prompt& a, const Batch& s, int w)
{
    int most = 0;
    int64_t all = 0;
    std::vector<int> count(a.batch);
    for (int b = 0; b < a.batch; ++b) {
        const bool any = start_of(s, b + 1) > start_of(s, b);
        const int len = s.lens[b] < a.at.limit ? s.lens[b] : a.at.limit;
        count[b] = any && len > 0 ? (len - 1) / kTileKeys + 1 : any;
        most = most > count[b] ? most : count[b];
        all += count[b];
    }
    int chunk = (int)((all + a.tiles - 1) / a.tiles);
    const int room = (most + a.parts - 1) / a.parts;
    chunk = chunk > room ? chunk : room;
    chunk = chunk > 1 ? chunk : 1;
    for (;; chunk += (chunk + 7) / 8) {
        int64_t held = 0;
        for (int n : count)
            held += (n + chunk - 1) / chunk;
        CHECK(held <= a.tiles || chunk < most);
        if (held <= a.tiles || chunk >= most)
            break;
    }
    for (int b = 0; b < a.batch; ++b) {
        const int own = (count[b] + chunk - 1) / chunk;
        if (w < own)
            return Part{b, w, own, chunk};
        w -= own;
    }
    return Part{0, 0, 0, 0};
}

static void check_map(const Prompt& a, const Batch& s, unsigned grid)
{
    std::map<std::tuple<int, int, int, int>, int> seen;
    std::map<int, std::pair<int, int>> split;   // parts and chunk of a sequence
    auto quotient = [](int x, int y) { return (int)((unsigned)x / (unsigned)y); };
    for (unsigned block = 0; block < grid; ++block) {
        int b, tile, part, parts = a.parts, chunk = a.chunk, kv;
        if (a.order == kShares) {
            const int w = (int)block / a.heads;
            const Part p = part_at(a, s, w);
            if (p.parts == 0)
                continue;
            b = p.b, tile = 0, part = p.part, parts = p.parts, chunk = p.chunk;
            kv = ((int)block - w * a.heads + part) % a.heads;
            CHECK(parts <= a.parts);
        } else {
            const Spot spot = spot_of(a, (int)block, quotient);
            CHECK(spot.kv >= 0 && spot.kv < a.heads && spot.part >= 0 && spot.part < a.parts && spot.place >= 0 && spot.place < a.tiles &&
                  spot.lap >= 0 && spot.lap < a.laps);
            kv = spot.kv, part = spot.part, tile = spot.place;
            if (a.order == kTogether) {
                b = 0;
                while (b + 1 < a.batch && (int64_t)start_of(s, b + 1) * a.group / kTileRows + b + 1 <= spot.place)
                    ++b;
                tile = spot.place - (int)((int64_t)start_of(s, b) * a.group / kTileRows) - b;
            } else {
                b = a.order == kSingle ? spot.place : spot.lap;
                tile = a.order == kSingle ? 0 : spot.place;
            }
        }
        CHECK(b >= 0 && b < a.batch);
        int n = start_of(s, b + 1) - start_of(s, b);
        n = n < a.max_new ? n : a.max_new;
        if (n <= 0 || tile < 0 || (int64_t)tile * kTileRows >= (int64_t)n * a.group)
            continue;
        ++seen[{kv, b, tile, part}];
        split[b] = {parts, chunk};
    }
    size_t expected = 0;
    for (int b = 0; b < a.batch; ++b) {
        int n = start_of(s, b + 1) - start_of(s, b);
        n = n < a.max_new ? n : a.max_new;
        if (n <= 0)
            continue;
        const int len = s.lens[b] < 0 ? 0 : s.lens[b] < a.at.limit ? s.lens[b] : a.at.limit;
        const auto [parts, chunk] = split[b];
        for (int tile = 0; (int64_t)tile * kTileRows < (int64_t)n * a.group; ++tile) {
            for (int kv = 0; kv < a.heads; ++kv)
                for (int part = 0; part < parts; ++part, ++expected)
                    CHECK((seen[{kv, b, tile, part}]) == 1);
            // every slot that a token of the tile sees is in a tile of keys that some part takes
            const int r0 = tile * kTileRows, r1 = (int)(r0 + kTileRows < (int64_t)n * a.group ? r0 + kTileRows : n * a.group) - 1;
            auto position = [&](int r) {
                const int p = len - n + r / a.group;
                return !a.causal ? kEverySlot : p > -1 ? p : -1;
            };
            const int lowest = position(r0), highest = position(r1);
            const int top = highest + 1 < len ? highest + 1 : len, all = top > 0 ? (top + kTileKeys - 1) / kTileKeys : 0;
            int jump = 0;
            if (a.window > 0 && lowest >= a.window) {
                jump = (lowest - a.window + 1) / kTileKeys - a.sink_tiles;
                jump = jump > 0 ? jump : 0;
            }
            CHECK((int64_t)parts * chunk >= all - jump);
            for (int r = r0; r <= r1; r += r + a.group <= r1 ? a.group : 1) {
                const int p = position(r);
                for (int k : {0, a.sinks - 1, p - a.window + 1, p, len - 1}) {
                    const bool sees = k >= 0 && k < len && k <= p && (a.window == 0 || k > p - a.window || k < a.sinks);
                    const int u = k / kTileKeys;
                    if (sees)
                        CHECK((u < a.sink_tiles || u >= a.sink_tiles + jump) && u < all);
                }
            }
        }
    }
    CHECK(seen.size() == expected);
}

static const uintptr_t kBase = uintptr_t(1) << 40;   // stands for device memory, which host code does not read

static void check_parts(const float* ms, const float* out, int64_t heads, int parts, int dim, size_t bytes)
{
    const uintptr_t m = reinterpret_cast<uintptr_t>(ms), o = reinterpret_cast<uintptr_t>(out), end = kBase + bytes;
    CHECK(m >= kBase && m % 16 == 0 && o % 16 == 0);
    CHECK(m + (uintptr_t)heads * parts * 8 <= end && o + (uintptr_t)heads * parts * dim * 4 <= end);
    CHECK(m + (uintptr_t)heads * parts * 8 <= o);
}

template <class T>
static T taken(const std::vector<unsigned char>& bytes)
{
    T t;
    memcpy(&t, bytes.data(), sizeof t);
    return t;
}

static gemv_kv_cache cache_of()
{
    gemv_kv_cache c{};
    c.k = reinterpret_cast<void*>(kBase);
    c.v = reinterpret_cast<void*>(kBase);
    c.dtype = pick({(int)GEMV_F16, (int)GEMV_BF16});
    c.pages = 1 << 20;
    c.page_size = pick({1, 5, 8, 16, 24, 64, 128});
    c.heads = pick({1, 1, 2, 3, 4, 5, 8, 16});
    c.head_dim = pick({8, 64, 80, 96, 128, 136, 256});
    c.stride_head = c.head_dim;
    c.stride_slot = (int64_t)c.heads * c.head_dim;
    c.stride_page = c.stride_slot * c.page_size;
    return c;
}

static Batch batch_of(int n, int most_new, int most_old, bool alike)
{
    Batch s;
    int row = below(3) == 0 ? below(200) : 0;
    s.starts.push_back(row);
    s.max_new = 1;
    for (int b = 0; b < n; ++b) {
        const int add = alike && b > 0 ? most_new - below(3) : b == 0 ? most_new : below(most_new + 1), fresh = add > 0 ? add : 0;
        s.max_new = s.max_new > fresh ? s.max_new : fresh;
        row += fresh;
        s.starts.push_back(row);
        s.lens.push_back(below(9) == 0 ? below(fresh + 1) : fresh + below(most_old + 1));
    }
    s.rows = row + (below(3) == 0 ? below(200) : 0);
    return s;
}

static gemv_kv_batch sequences(const gemv_kv_cache& c, const Batch& s, int spare)
{
    int longest = 1;
    for (int n : s.lens)
        longest = longest > n ? longest : n;
    gemv_kv_batch q{};
    q.table = reinterpret_cast<const int32_t*>(kBase);
    q.width = (longest + c.page_size - 1) / c.page_size + spare;
    q.table_stride = q.width;
    q.lens = reinterpret_cast<const int32_t*>(kBase);   // the copies of the checks are on the host
    q.batch = (int)s.lens.size();
    q.max_len = below(2) ? longest : 0x7FFFFFFF;
    return q;
}

static void prompts()
{
    const gemv_kv_cache c = cache_of();
    const int group = pick({1, 1, 2, 4, 5, 7, 8, 16, 130});
    const int n = pick({1, 2, 3, 7, 64, 65, 100}), few = pick({2, 7, 40}), many = pick({300, 1500, 5000});
    Batch s = batch_of(n, n > 10 || below(2) ? few : many, pick({0, 50, 3000, 60000}), below(2) == 0);
    if ((int64_t)s.rows * group * c.heads > 400000)
        return;
    const gemv_kv_batch q = sequences(c, s, below(2) ? 0 : 700);
    const int heads = c.heads * group, window = below(3) == 0 ? 1 + below(3000) : 0, sinks = window ? pick({0, 1, 4, 64, 100, 5000}) : 0;
    int max_new = s.max_new < 2 ? 2 : s.max_new;
    if (below(4) == 0)
        max_new = s.rows > 1 ? s.rows + below(2) : 2;
    if (below(6) == 0)
        max_new = 2 + below(max_new);   // older rows are left out
    void* base = reinterpret_cast<void*>(kBase);
    const size_t need = gemv_prompt_attention_workspace(&c, &q, s.rows, max_new, heads, window, sinks);
    const int64_t stride = (int64_t)heads * c.head_dim;
    auto call = [&](size_t bytes) {
        launches.clear();
        sizes[0] = sizeof(Prompt), sizes[1] = 0;
        return gemv_prompt_attention(&c, &q, reinterpret_cast<const int32_t*>(kBase), s.rows, max_new, base, stride, heads, 0.1f, window, sinks,
                                     base, need ? base : nullptr, bytes, nullptr);
    };
    if (need > 0)
        CHECK(call(need - 1) == GEMV_E_INVAL && launches.empty());
    CHECK(call(need) == GEMV_OK && launches.size() == (need > 0 ? 2u : 1u));
    if (launches.empty())
        return;
    const Prompt a = taken<Prompt>(launches[0].first);
    CHECK(launches[0].block == 256u * outputs_of(c.head_dim));
    if (launches[0].grid > 20000)
        return;
    check_map(a, s, launches[0].grid);
    CHECK((a.part_out != nullptr) == (need > 0) && (need > 0 || a.parts == 1));
    if (need > 0)
        check_parts(a.part_ms, a.part_out, (int64_t)s.rows * heads, a.parts, c.head_dim, need);
}

static void prefixes()
{
    const gemv_kv_cache c = cache_of();
    const int group = pick({1, 2, 4, 5, 8, 16, 130}), heads = c.heads * group;
    Batch far = batch_of(pick({1, 2, 5}), pick({1, 3, 16, 64}), pick({0, 100, 30000}), below(2) == 0);
    Batch near;
    near.rows = far.rows > 0 ? far.rows : 1;
    far.rows = near.rows;
    far.max_new = near.rows;
    for (int b = 0; b < near.rows; ++b)
        near.lens.push_back(below(4) == 0 ? 0 : below(1000));
    if ((int64_t)near.rows * heads > 100000)
        return;
    const gemv_kv_batch f = sequences(c, far, below(3)), q = sequences(c, near, below(3));
    void* base = reinterpret_cast<void*>(kBase);
    const size_t need = gemv_prefix_attention_workspace(&c, &f, &q, heads);
    launches.clear();
    sizes[0] = sizeof(Prompt), sizes[1] = sizeof(Attention);
    auto call = [&](size_t bytes) {
        return gemv_prefix_attention(&c, &f, reinterpret_cast<const int32_t*>(kBase), &q, base, (int64_t)heads * c.head_dim, heads, 0.1f, base,
                                     base, bytes, nullptr);
    };
    CHECK(need > 0 && call(need - 1) == GEMV_E_INVAL && launches.empty());
    CHECK(call(need) == GEMV_OK && launches.size() == 2);
    if (launches.size() != 2)
        return;
    const Launch& l = launches[0];
    const Prompt a = taken<Prompt>(l.first);
    const Attention own = taken<Attention>(l.second);
    CHECK(l.blocks % 8 == 0 && l.blocks >= l.count && l.blocks - l.count < 8 && l.grid >= (unsigned)l.blocks);
    if (l.count > 0 && l.count < 20000) {
        check_map(a, far, (unsigned)l.count);
        check_parts(a.part_ms, a.part_out, (int64_t)near.rows * heads, a.parts, c.head_dim, need);
    }
    CHECK((int64_t)own.parts * own.chunk >= own.at.limit && own.chunk <= kMaxChunk && own.chunk % 64 == 0);
    CHECK(l.grid - l.blocks >= (unsigned)(own.heads * own.batch * own.parts * own.tiles));
    check_parts(own.part_ms, own.part_out, (int64_t)near.rows * heads, own.parts, c.head_dim, need);
}

// single tokens through a window: what they see is covered by the parts
static void newest_tokens()
{
    const gemv_kv_cache c = cache_of();
    Batch s = batch_of(pick({1, 5, 64}), 1, pick({10, 3000, 60000}), true);
    const gemv_kv_batch q = sequences(c, s, below(100));
    const int heads = c.heads * pick({1, 4, 17}), window = 1 + below(pick({20, 5000, 70000})), sinks = pick({0, 4, 1000});
    void* base = reinterpret_cast<void*>(kBase);
    const size_t need = gemv_prompt_attention_workspace(&c, &q, q.batch, 1, heads, window, sinks);
    launches.clear();
    sizes[0] = sizeof(Attention), sizes[1] = 0;
    CHECK(gemv_prompt_attention(&c, &q, nullptr, q.batch, 1, base, (int64_t)heads * c.head_dim, heads, 0.1f, window, sinks, base,
                                need ? base : nullptr, need, nullptr) == GEMV_OK);
    if (launches.empty())
        return;
    const Attention a = taken<Attention>(launches[0].first);
    for (int len : s.lens) {
        len = len < a.at.limit ? len : a.at.limit;
        if (a.window > 0 && len > a.window) {
            const int low = len - a.window, gap = (low & ~15) - a.sinks16;
            len -= gap > 0 ? gap : 0;
        }
        CHECK((int64_t)a.parts * a.chunk >= len);
    }
    if (need > 0)
        check_parts(a.part_ms, a.part_out, (int64_t)q.batch * heads, a.parts, c.head_dim, need);
}

// numbers of any size: whatever the status, nothing overflows on the way
static int wild()
{
    switch (below(6)) {
    case 0: return below(4) - 2;
    case 1: return 0x7FFFFFFF - below(3);
    case 2: return (int)(0x80000000u + next() % 3);
    case 3: return below(300);
    default: return (int)(next() >> below(31));
    }
}

static int64_t wide() { return below(3) == 0 ? (int64_t)wild() * wild() / 8 * 8 : (int64_t)wild() * 8; }

static void any_numbers()
{
    gemv_kv_cache c = cache_of();
    if (below(2)) {
        c.pages = wild(), c.page_size = wild(), c.heads = wild(), c.head_dim = below(2) ? 8 * below(33) : wild();
        c.stride_page = wide(), c.stride_slot = wide(), c.stride_head = wide();
    }
    gemv_kv_batch q{reinterpret_cast<const int32_t*>(kBase), wide(), wild(), reinterpret_cast<const int32_t*>(kBase), wild(), wild()}, f = q;
    if (below(2))
        q.table_stride = q.width, f.batch = wild(), f.table_stride = f.width = wild();
    void* base = reinterpret_cast<void*>(kBase);
    const int32_t* ints = reinterpret_cast<const int32_t*>(kBase);
    const int rows = wild(), max_new = wild(), heads = wild(), window = wild(), sinks = wild();
    launches.clear();
    sizes[0] = sizes[1] = 0;
    (void)gemv_prompt_attention_workspace(&c, &q, rows, max_new, heads, window, sinks);
    (void)gemv_prefix_attention_workspace(&c, &f, &q, heads);
    (void)gemv_prompt_attention(&c, &q, ints, rows, max_new, base, wide(), heads, 0.5f, window, sinks, base, base, ~size_t(0), nullptr);
    (void)gemv_prefix_attention(&c, &f, ints, &q, base, wide(), heads, 0.5f, base, base, ~size_t(0), nullptr);
    gemv_page_pool p{reinterpret_cast<int32_t*>(kBase), ints, wild(), wild(), reinterpret_cast<int32_t*>(2 * kBase), wide(), wild(), wild()};
    int32_t* out = reinterpret_cast<int32_t*>(4 * kBase);
    (void)gemv_reserve_pages(&p, ints, ints, rows, out, out, out, out, reinterpret_cast<int64_t*>(out), nullptr);
    (void)gemv_release_pages_workspace(&p);
    (void)gemv_release_pages(&p, ints, out, base, ~size_t(0), nullptr);
    gemv_rotation how{below(2) ? 8 * below(33) : wild(), 2 * below(129), below(2), reinterpret_cast<const double*>(kBase), below(2), 1e-6f, below(4)};
    gemv_heads h[3];
    for (gemv_heads& x : h)
        x = gemv_heads{base, wide(), below(2) ? below(40) : wild(), below(2) ? base : nullptr, reinterpret_cast<void*>(kBase * (1 + below(3))), wide()};
    (void)gemv_norm_rotate(&how, &h[0], below(2) ? &h[1] : nullptr, below(3), below(3), ints, rows, nullptr);
    (void)gemv_norm_rotate_append(&how, &h[0], &h[1], &h[2], below(3), ints, rows, &c, reinterpret_cast<const int64_t*>(kBase), nullptr);
    for (const Launch& l : launches)
        CHECK(l.grid > 0 && (uint64_t)l.grid * l.block <= (uint64_t)gemv_device::kMaxWorkItems);
}

int main()
{
    for (int chip : {256, 80}) {
        cus = chip;
        for (int i = 0; i < 400; ++i, ++trial)
            prompts();
        for (int i = 0; i < 200; ++i, ++trial)
            prefixes();
        for (int i = 0; i < 400; ++i, ++trial)
            newest_tokens();
        for (int i = 0; i < 6000; ++i, ++trial)
            any_numbers();
    }
    if (failures == 0)
        printf("%ld trials: every launch covers its work\n", trial);
    return failures == 0 ? 0 : 1;
}
