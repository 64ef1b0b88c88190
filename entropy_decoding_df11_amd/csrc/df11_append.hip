// Keys and values of new tokens into a paged cache, rotated on the way, and
// their queries rotated (gfx950).
//
//   (a, b) -> (a cos - b sin, b cos + a sin)     in float, rounded once
//
// Every element is read once and written once.  A thread has one unit of a
// token: eight rotated pairs (16 elements), or eight elements that are copied,
// all in 16-byte accesses; a workgroup's units belong to one token, so that
// what finds its place (sequence, page) is the same for all of its lanes.  The
// elements are asked for before that chain (starts, length, page) is followed.
//
// Few tokens are bound by the chain, four loads that wait for each other: one token
// of 32 + 8 + 8 heads of 128 takes 3.2 us (the call from Python 15).  Many are bound
// by memory: 1536 tokens of float sums 11.3 us (4.0 TB/s of 45 MB), 9400 of FP16
// with neighbouring pairs 56 us (4.1 TB/s of 232 MB; with two accesses of 16 bytes
// side by side a lane, which leave every other chunk to the next access, 69).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <type_traits>

#include <stdint.h>

#include "df11.h"
#include "df11_attention_plan.h"
#include "df11_device.h"
#include "df11_kv.h"
#include "df11_types.h"

namespace {

struct Rows {
    const void *p;
    uint64_t stride, head_stride;
};

struct AppendArgs {
    df11::KvBatch b;
    df11::KvPages k_pages, v_pages;
    Rows k, v, q;
    void *q_out;
    uint64_t q_out_stride, q_out_head_stride;
    const float *rotary;
    const int32_t *positions;
    uint64_t rotary_rows;
    uint32_t n_pages, page_size;
    uint32_t q_heads, kv_heads, dim, rotary_dims;
    uint32_t units_head;  // units of a rotated head, of a copied one
    uint32_t units_copy;
    uint32_t units;       // of a token
    uint32_t head_magic, copy_magic;    // floor(2^32 / units_head) + 1, 0 for one unit
    uint32_t page_magic, page_shift;    // df11::page_of
};

// N consecutive elements as floats and back (N * 2 or 16 bytes aligned).
template <typename T, int N>
__device__ __forceinline__ void load_unit(const T *p, float (&f)[N]) {
    if constexpr (sizeof(T) * N > 16) {
#pragma unroll
        for (int i = 0; i < N; i += 4) load_vec<T, 4>(p + i, *reinterpret_cast<float(*)[4]>(&f[i]));
    } else {
        load_vec<T, N>(p, f);
    }
}

// N pairs rotated in place, x and y their first and second elements.
template <int N>
__device__ __forceinline__ void turn(float (&x)[N], float (&y)[N], const float (&c)[N], const float (&s)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float a = x[i], b = y[i];
        x[i] = a * c[i] - b * s[i];
        y[i] = b * c[i] + a * s[i];
    }
}

// N: pairs of a rotated unit and elements of a copied one.  kNext: neighbouring
// pairs, of which a rotated unit has N / 2 (or one): then lanes read and write next to
// each other in every access.
template <typename IN, typename OUT, int N, bool kNext>
__global__ __launch_bounds__(256) void df11_append_kernel(AppendArgs a) {
    const uint32_t token = blockIdx.x, unit = min(blockIdx.y * blockDim.x + threadIdx.x, a.units - 1u);
    const uint32_t q_units = a.q_heads * a.units_head, k_units = a.kv_heads * a.units_head;
    const bool mine = blockIdx.y * blockDim.x + threadIdx.x < a.units;
    // What the unit reads, of q, k or v.
    const uint32_t kind = unit < q_units ? 0u : unit < q_units + k_units ? 1u : 2u;
    const uint32_t u = unit - (kind == 0u ? 0u : kind == 1u ? q_units : q_units + k_units);
    // (a unit's number times the units of a head is far below 2^32: the quotient by
    // the multiplication is exact)
    const uint32_t magic = kind == 2u ? a.copy_magic : a.head_magic;
    const uint32_t head = magic ? __umulhi(u, magic) : u;
    const uint32_t part = u - head * (kind == 2u ? a.units_copy : a.units_head);
    const Rows &r = kind == 0u ? a.q : kind == 1u ? a.k : a.v;
    const IN *from = static_cast<const IN *>(r.p) + token * r.stride + head * r.head_stride;
    // Its elements d0 .. and, of a rotated one of pairs that lie apart, d1 ..
    constexpr uint32_t kPairs = kNext && N > 1 ? N / 2 : N;  // of a rotated unit
    const uint32_t half = a.rotary_dims / 2u, turned = half / kPairs;
    const bool turns = kind != 2u && part < turned;
    const uint32_t d0 = turns ? (kNext ? 2u : 1u) * part * kPairs
                              : (kind == 2u ? part * N : a.rotary_dims + (part - turned) * N);
    const uint32_t d1 = kNext ? d0 + 1u : d0 + half;
    constexpr bool kTwo = !kNext || N == 1;  // a rotated unit has two accesses
    float x[N], y[N];
    load_unit(from + d0, x);
    if (kTwo && turns) load_unit(from + d1, y);
    // Where it goes.
    const int64_t at = a.positions ? a.positions[token] : 0;
    const int32_t seq = __builtin_amdgcn_readfirstlane(sequence_of(a.b, static_cast<int32_t>(token)));
    if (seq < 0 || !mine) return;
    const int64_t length = a.b.lengths[seq];
    const int64_t place = length + (static_cast<int64_t>(token) - a.b.starts[seq]);
    OUT *to;
    if (kind == 0u) {
        to = static_cast<OUT *>(a.q_out) + token * a.q_out_stride + head * a.q_out_head_stride;
    } else {
        if (length < 0 || place < 0 || place >= static_cast<int64_t>(a.b.table_pages) * a.page_size) return;
        const uint32_t p = static_cast<uint32_t>(place), page = df11::page_of(p, a.page_magic, a.page_shift);
        const uint32_t id = static_cast<uint32_t>(a.b.page_table[seq * a.b.table_stride + page]);
        if (id >= a.n_pages) return;
        const df11::KvPages &c = kind == 1u ? a.k_pages : a.v_pages;
        to = static_cast<OUT *>(c.p) + id * c.page_stride + (p - page * a.page_size) * c.place_stride + head * c.head_stride;
    }
    if (turns) {
        const int64_t position = a.positions ? at : place;
        const bool known = position >= 0 && static_cast<uint64_t>(position) < a.rotary_rows;
        const float *row = a.rotary + (known ? position : 0) * a.rotary_dims + part * kPairs;
        float c[kPairs], s[kPairs];
        load_unit(row, c);
        load_unit(row + half, s);
        if (!known) {
#pragma unroll
            for (uint32_t i = 0; i < kPairs; ++i) c[i] = s[i] = __builtin_nanf("");
        }
        if constexpr (kTwo) {
            turn(x, y, c, s);
            store_vec<OUT, N>(to + d1, y);
        } else {
            float first[kPairs], second[kPairs];
#pragma unroll
            for (uint32_t i = 0; i < kPairs; ++i) {
                first[i] = x[2 * i];
                second[i] = x[2 * i + 1];
            }
            turn(first, second, c, s);
#pragma unroll
            for (uint32_t i = 0; i < kPairs; ++i) {
                x[2 * i] = first[i];
                x[2 * i + 1] = second[i];
            }
        }
    }
    store_vec<OUT, N>(to + d0, x);
}

template <typename IN, typename OUT>
const void *pick_width(bool wide, bool next) {
    if (next)
        return wide ? reinterpret_cast<const void *>(&df11_append_kernel<IN, OUT, 8, true>)
                    : reinterpret_cast<const void *>(&df11_append_kernel<IN, OUT, 1, true>);
    return wide ? reinterpret_cast<const void *>(&df11_append_kernel<IN, OUT, 8, false>)
                : reinterpret_cast<const void *>(&df11_append_kernel<IN, OUT, 1, false>);
}

template <typename OUT>
const void *pick_in(uint32_t dtype, bool wide, bool next) {
    return dtype == DF11_FP32   ? pick_width<float, OUT>(wide, next)
           : dtype == DF11_BF16 ? pick_width<bf16_t, OUT>(wide, next)
                                : pick_width<fp16_t, OUT>(wide, next);
}

}  // namespace

extern "C" int df11_append_kv(const df11_kv_cache *c, const df11_kv_batch *b, const df11_append *given, void *hip_stream) {
    uint64_t k_span = 0, v_span = 0;
    const int rc = check_kv(c, b, k_span, v_span);
    if (rc) return rc;
    if (!given) return DF11_E_INVALID_ARG;
    df11_append used = *given;
    for (uint64_t *s : {&used.k_stride, &used.v_stride, &used.q_stride, &used.q_out_stride}) *s = kv_stride(b->n_tokens, *s);
    for (uint64_t *s : {&used.k_head_stride, &used.v_head_stride}) *s = kv_stride(c->heads, *s);
    for (uint64_t *s : {&used.q_head_stride, &used.q_out_head_stride}) *s = kv_stride(used.q_heads, *s);
    const df11_append *a = &used;
    const uint32_t bytes = dtype_bytes(a->dtype), dim = c->head_dim, tokens = b->n_tokens;
    // (tensors without elements have no address, whatever their heads)
    if (!bytes || !a->q != !a->q_out || (a->q ? !a->q_heads || a->q_heads > kMaxKvHeads : a->q_heads != 0 && tokens))
        return DF11_E_INVALID_ARG;
    if (a->rotary && (a->rotary_dims < 2 || a->rotary_dims % 2 || a->rotary_dims > dim || !aligned(a->rotary, 4) ||
                      a->rotary_rows > (1ull << 40) || a->interleaved > 1))
        return DF11_E_INVALID_ARG;
    if (a->positions && !aligned(a->positions, 4)) return DF11_E_INVALID_ARG;
    if (tokens == 0 || b->n_seqs == 0) return DF11_OK;
    if (!a->k || !a->v) return DF11_E_INVALID_ARG;
    // Places that lie on each other would hold what was written last.
    const Runs k_runs = kv_runs(c->k, c->k_page_stride, c->k_place_stride, c->k_head_stride, *c);
    const Runs v_runs = kv_runs(c->v, c->v_page_stride, c->v_place_stride, c->v_head_stride, *c);
    if (!k_runs.nested || !v_runs.nested || !lie_apart(k_runs, v_runs)) return DF11_E_INVALID_ARG;
    if (a->rotary && !a->rotary_rows) return DF11_E_INVALID_ARG;
    const uint32_t rotary_dims = a->rotary ? a->rotary_dims : 0;
    struct In {
        const void *p;
        uint64_t stride, head_stride, heads;
    } ins[] = {{a->q, a->q_stride, a->q_head_stride, a->q_heads},
               {a->k, a->k_stride, a->k_head_stride, c->heads},
               {a->v, a->v_stride, a->v_head_stride, c->heads}};
    bool wide = rotary_dims % 16 == 0 && aligned(a->rotary, 16) && aligned(a->q_out, 16) && a->q_out_stride % 8 == 0 && a->q_out_head_stride % 8 == 0;
    Runs in_runs[3];
    const auto runs = [&](const void *p, uint64_t stride, uint64_t heads, uint64_t head_stride, uint64_t size) {
        return runs_of(p, size * dim, {{tokens, size * stride}, {heads, size * head_stride}});
    };
    for (int i = 0; i < 3; ++i) {
        if (ins[i].stride >= kMaxKvStride || ins[i].head_stride >= (1ull << 32) || !aligned(ins[i].p, bytes))
            return DF11_E_INVALID_ARG;
        in_runs[i] = runs(ins[i].p, ins[i].stride, ins[i].heads, ins[i].head_stride, bytes);
        wide = wide && aligned(ins[i].p, 16) && ins[i].stride % 8 == 0 && ins[i].head_stride % 8 == 0;
    }
    // The cache's halves, q_out and everything that is read lie apart; q_out
    // may lie exactly on q, beside k and v in the rows of one tensor.
    const uint64_t q_out_span = a->q ? 2 * kv_span(tokens, a->q_out_stride, a->q_heads, a->q_out_head_stride, dim) : 0;
    if (a->q && (!aligned(a->q_out, 2) || a->q_out_stride >= kMaxKvStride || a->q_out_head_stride >= (1ull << 32) ||
                 !kv_apart(tokens, a->q_out_stride, a->q_heads, a->q_out_head_stride, dim)))
        return DF11_E_INVALID_ARG;
    const bool on_q = a->q && a->q == a->q_out && a->q_stride == a->q_out_stride &&
                      a->q_head_stride == a->q_out_head_stride && a->dtype == c->dtype;
    const void *outs[] = {c->k, c->v, a->q_out};
    const uint64_t out_spans[] = {k_span, v_span, q_out_span};
    const Runs out_runs[] = {k_runs, v_runs, runs(a->q_out, a->q_out_stride, a->q_heads, a->q_out_head_stride, 2)};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 3; ++j) {
            if (!lie_apart(out_runs[i], in_runs[j]) && !(i == 2 && j == 0 && on_q)) return DF11_E_INVALID_ARG;
            if (i == 2 && j < 2 && !lie_apart(out_runs[i], out_runs[j])) return DF11_E_INVALID_ARG;
        }
        if (!clear_of_batch(*b, outs[i], out_spans[i]) ||
            overlaps(outs[i], out_spans[i], a->rotary, 4 * a->rotary_rows * rotary_dims) ||
            overlaps(outs[i], out_spans[i], a->positions, a->positions ? 4ull * tokens : 0))
            return DF11_E_INVALID_ARG;
    }
    AppendArgs k{};
    k.b = kernel_batch(*b);
    k.k_pages = kernel_pages(c->k, c->k_page_stride, c->k_place_stride, c->k_head_stride, *c);
    k.v_pages = kernel_pages(c->v, c->v_page_stride, c->v_place_stride, c->v_head_stride, *c);
    k.q = Rows{a->q, a->q_stride, a->q_head_stride};
    k.k = Rows{a->k, a->k_stride, a->k_head_stride};
    k.v = Rows{a->v, a->v_stride, a->v_head_stride};
    k.q_out = a->q_out;
    k.q_out_stride = a->q_out_stride;
    k.q_out_head_stride = a->q_out_head_stride;
    k.rotary = a->rotary;
    k.positions = a->positions;
    k.rotary_rows = a->rotary_rows;
    k.n_pages = c->n_pages;
    k.page_size = c->page_size;
    k.q_heads = a->q_heads;
    k.kv_heads = c->heads;
    k.dim = dim;
    k.rotary_dims = rotary_dims;
    const bool next = a->interleaved != 0 && rotary_dims;
    const uint32_t each = wide ? 8 : 1, pairs = wide && next ? 4 : each;
    k.units_head = rotary_dims / 2 / pairs + (dim - rotary_dims) / each;
    k.units_copy = dim / each;
    // (at most 4096 heads of 256 elements, three times)
    k.units = (a->q_heads + c->heads) * k.units_head + c->heads * k.units_copy;
    const auto magic = [](uint32_t n) { return n > 1 ? static_cast<uint32_t>((1ull << 32) / n + 1u) : 0u; };
    k.head_magic = magic(k.units_head);
    k.copy_magic = magic(k.units_copy);
    k.page_shift = df11::page_shift(c->page_size);
    k.page_magic = df11::page_magic(c->page_size, k.page_shift);
    (void)hipGetLastError();
    void *params[] = {&k};
    // (a dimension of a launch has fewer than 2^32 threads)
    const uint32_t threads = k.units >= 256 && tokens < kMaxKvTokens ? 256 : 64;
    static_assert(64ull * kMaxKvTokens < (1ull << 32) && 256ull * (kMaxKvTokens - 1) < (1ull << 32), "a launch holds it");
    return launch_kernel(c->dtype == DF11_BF16 ? pick_in<bf16_t>(a->dtype, wide, next)
                                              : pick_in<fp16_t>(a->dtype, wide, next),
                         dim3(tokens, (k.units + threads - 1) / threads), dim3(threads), params, 0,
                         static_cast<hipStream_t>(hip_stream), nullptr, nullptr);
}
