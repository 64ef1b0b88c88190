// The paged cache and its batch as the kernels that append to it and read it
// see them, and the checks that both entry points share.
#pragma once

#include <hip/hip_runtime.h>

#include <initializer_list>
#include <utility>

#include <stdint.h>

#include "df11.h"
#include "df11_device.h"
#include "df11_types.h"

namespace df11 {

// Kernel arguments of a batch (df11_kv_batch with its checks done).
struct KvBatch {
    const int32_t *starts, *lengths, *page_table;
    uint64_t table_stride;
    uint32_t n_seqs, table_pages, n_tokens;
};

// One of the cache's two halves.
struct KvPages {
    void *p;
    uint64_t page_stride, place_stride, head_stride;
};

}  // namespace df11

namespace {

constexpr uint64_t kMaxKvStride = 1ull << 40;
constexpr uint32_t kMaxKvTokens = 1u << 24;
constexpr uint32_t kMaxKvHeads = 4096;
constexpr uint64_t kMaxKvPlaces = 1ull << 30;  // of a sequence's pages

// Sequence of a token, the same in every lane, or -1: the last one that starts
// at the token or before.  All starts are compared at once, 64 at a time; a
// search would wait for one load after the other.
__device__ __forceinline__ int32_t sequence_of(const df11::KvBatch &b, int32_t token) {
    const uint32_t lane = threadIdx.x & (kWaveSize - 1);
    uint32_t before = 0;
    for (uint32_t at = 0; at < b.n_seqs; at += kWaveSize) {
        const bool in = at + lane < b.n_seqs && b.starts[at + lane] <= token;
        before += static_cast<uint32_t>(__popcll(__ballot(in)));
    }
    return before && token < b.starts[b.n_seqs] ? static_cast<int32_t>(before) - 1 : -1;
}

// Elements from the first to behind the last of a tensor of rows x heads x dim.
[[maybe_unused]] uint64_t kv_span(uint64_t rows, uint64_t stride, uint64_t heads, uint64_t head_stride, uint64_t dim) {
    return rows && heads ? (rows - 1) * stride + (heads - 1) * head_stride + dim : 0;
}

// A stride as it is used: along one element not at all.
[[maybe_unused]] uint64_t kv_stride(uint64_t count, uint64_t stride) { return count > 1 ? stride : 0; }

// Whether rows and heads of such a tensor lie apart (the larger stride steps
// over all that the smaller one reaches).
[[maybe_unused]] bool kv_apart(uint64_t rows, uint64_t stride, uint64_t heads, uint64_t head_stride, uint64_t dim) {
    if (rows <= 1 && heads <= 1) return true;
    if (heads <= 1) return stride >= dim;
    if (rows <= 1) return head_stride >= dim;
    return (head_stride >= dim && stride >= (heads - 1) * head_stride + dim) ||
           (stride >= dim && head_stride >= (rows - 1) * stride + dim);
}

// A tensor in memory as runs of `run` bytes along up to three dimensions, the largest
// stride first, in bytes; dimensions of one element or without a stride left out.
struct Runs {
    uintptr_t at;
    uint64_t run, span;  // span: from the first byte to behind the last
    uint64_t stride[3], count[3];
    int dims;
    bool nested;  // every stride steps over all that the smaller ones reach: no run lies on another
};

[[maybe_unused]] Runs runs_of(const void *p, uint64_t run, std::initializer_list<std::pair<uint64_t, uint64_t>> dims) {
    Runs r{reinterpret_cast<uintptr_t>(p), run, run, {}, {}, 0, true};
    for (const auto &[count, stride] : dims) {
        if (count <= 1) continue;
        if (stride == 0) {
            r.nested = false;
            continue;
        }
        int i = r.dims++;
        for (; i > 0 && r.stride[i - 1] < stride; --i) {
            r.stride[i] = r.stride[i - 1];
            r.count[i] = r.count[i - 1];
        }
        r.stride[i] = stride;
        r.count[i] = count;
    }
    for (int i = r.dims; i-- > 0;) {
        r.nested = r.nested && r.stride[i] >= r.span;
        r.span += (r.count[i] - 1) * r.stride[i];
    }
    return r;
}

// Whether two tensors are seen to share no byte: their spans lie apart, or, stepping
// alike along their outermost dimensions, no two of their steps do (parts of one
// tensor's rows, as a fused product leaves them).
[[maybe_unused]] bool lie_apart(const Runs &a, const Runs &b) {
    if (!a.at || !b.at || !a.span || !b.span || a.at + a.span <= b.at || b.at + b.span <= a.at) return true;
    if (!a.nested || !b.nested || !a.dims || !b.dims || a.stride[0] != b.stride[0]) return false;
    const auto inner = [](const Runs &r) {
        Runs in = r;
        in.span -= (r.count[0] - 1) * r.stride[0];
        --in.dims;
        for (int i = 0; i < in.dims; ++i) {
            in.stride[i] = r.stride[i + 1];
            in.count[i] = r.count[i + 1];
        }
        return in;
    };
    // A step of either reaches less than the stride: only those matter whose first
    // bytes are nearer than that.
    const int64_t stride = static_cast<int64_t>(a.stride[0]), off = static_cast<int64_t>(b.at - a.at);
    const Runs x = inner(a);
    Runs y = inner(b);
    for (int64_t n = -off / stride - 1; n <= -off / stride + 1; ++n) {
        // (n: b's step over a's)
        if (n <= -static_cast<int64_t>(a.count[0]) || n >= static_cast<int64_t>(b.count[0])) continue;
        y.at = b.at + static_cast<uint64_t>(n * stride);
        if (!lie_apart(x, y)) return false;
    }
    return true;
}

// Pages x places x heads of one half of the cache, `span` receiving its bytes.
[[maybe_unused]] bool kv_pages_ok(const void *p, uint64_t page, uint64_t place, uint64_t head, const df11_kv_cache &c,
                                  uint64_t &span) {
    if (!p || !aligned(p, 16)) return false;
    const uint64_t strides[] = {page, place, head}, counts[] = {c.n_pages, c.page_size, c.heads};
    span = c.head_dim;
    for (int i = 0; i < 3; ++i) {
        if (counts[i] == 1) continue;
        if (strides[i] % 8 || strides[i] >= kMaxKvStride) return false;
        // (2^31 pages of strides below 2^40 would pass 64 bits in bytes)
        if (strides[i] > (1ull << 60) / counts[i]) return false;
        span += (counts[i] - 1) * strides[i];
    }
    span *= 2;
    return true;
}

// Checks of the cache and the batch; the spans of k and v in bytes.
[[maybe_unused]] int check_kv(const df11_kv_cache *c, const df11_kv_batch *b, uint64_t &k_span, uint64_t &v_span) {
    if (!c || !b) return DF11_E_INVALID_ARG;
    if ((c->dtype != DF11_BF16 && c->dtype != DF11_FP16) || !c->n_pages || c->n_pages > 0x7FFFFFFFu || !c->page_size ||
        c->page_size > (1u << 20) || !c->heads || c->heads > kMaxKvHeads || c->head_dim < 8 || c->head_dim % 8 ||
        c->head_dim > DF11_MAX_HEAD_DIM)
        return DF11_E_INVALID_ARG;
    if (!kv_pages_ok(c->k, c->k_page_stride, c->k_place_stride, c->k_head_stride, *c, k_span) ||
        !kv_pages_ok(c->v, c->v_page_stride, c->v_place_stride, c->v_head_stride, *c, v_span))
        return DF11_E_INVALID_ARG;
    if (b->n_tokens > kMaxKvTokens || b->n_seqs > kMaxKvTokens || b->table_stride >= kMaxKvStride ||
        static_cast<uint64_t>(b->table_pages) * c->page_size > kMaxKvPlaces)
        return DF11_E_INVALID_ARG;
    if (!b->starts || !aligned(b->starts, 4)) return DF11_E_INVALID_ARG;
    if (b->n_seqs && (!b->lengths || !aligned(b->lengths, 4))) return DF11_E_INVALID_ARG;
    if (b->n_seqs && b->table_pages && (!b->page_table || !aligned(b->page_table, 4))) return DF11_E_INVALID_ARG;
    return DF11_OK;
}

// Whether an output of `bytes` at p lies clear of the batch's arrays.
[[maybe_unused]] bool clear_of_batch(const df11_kv_batch &b, const void *p, uint64_t bytes) {
    const uint64_t table = b.n_seqs && b.table_pages ? 4 * ((b.n_seqs - 1) * b.table_stride + b.table_pages) : 0;
    return !overlaps(p, bytes, b.starts, 4ull * (b.n_seqs + 1)) && !overlaps(p, bytes, b.lengths, 4ull * b.n_seqs) &&
           !overlaps(p, bytes, b.page_table, table);
}

// One half of the cache as runs.
[[maybe_unused]] Runs kv_runs(const void *p, uint64_t page, uint64_t place, uint64_t head, const df11_kv_cache &c) {
    return runs_of(p, 2ull * c.head_dim, {{c.n_pages, 2 * page}, {c.page_size, 2 * place}, {c.heads, 2 * head}});
}

[[maybe_unused]] df11::KvPages kernel_pages(void *p, uint64_t page, uint64_t place, uint64_t head, const df11_kv_cache &c) {
    return df11::KvPages{p, kv_stride(c.n_pages, page), kv_stride(c.page_size, place), kv_stride(c.heads, head)};
}

[[maybe_unused]] df11::KvBatch kernel_batch(const df11_kv_batch &b) {
    return df11::KvBatch{b.starts, b.lengths, b.page_table, b.table_stride, b.n_seqs, b.table_pages, b.n_tokens};
}

}  // namespace
