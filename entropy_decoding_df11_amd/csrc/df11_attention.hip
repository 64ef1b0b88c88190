// Attention of a batch's new tokens over a paged cache (gfx950).
//
//   out = sum over the visible places j of p_j v_j,  p = softmax(scale q . k_j)
//
// in one pass over the places, with the softmax's running maximum and sum: for
// a row's reference m, w_j = 2^(c (s_j - m)) with c = scale log2(e), and what
// has been summed is multiplied by 2^(c (m - m')) when the reference moves to
// m'.  It moves only where a weight passes what the type has room for, so that
// blocks without a new maximum need nothing across lanes.  BF16 has float's range:
// references are the largest score, weights pass them by 2^8 at most, and a weight's
// relative rounding depends on nothing.  FP16 loses bits of a weight below 2^-14 and
// the weight below 2^-25: references lie 2^7 below the largest score and weights
// reach 2^15, so that weights keep their precision down to 2^-21 of the largest
// score's when the reference was taken, and from there on are off by 2^-32 of it at
// most.  (Without the 2^7 a place 17 nats ahead left what others alike had added
// off by 44%.)
//
// One rounding of a weight puts outputs off by 0.0020 to 0.0023 of their norm in BF16,
// where rounding the result alone gives 0.0017.  A second product with the weights'
// remainders would leave the latter: nothing slower for few rows, but prompts'
// pieces 196 -> 237 us, the tree below 184 -> 231 and trees of a batch 47 -> 55.
//
// A query head's rows of one key head are the columns of the products, so that
// all heads of a group read a place once:
//   S^T = K Q^T    v_mfma_f32_16x16x32: lane l holds places 4 (l / 16) .. + 3 of
//                  a 16-place tile for row l mod 16
//   O^T = V^T W^T  of two place tiles at once, with the places in the order in
//                  which S^T left them (4 (l / 16) .. + 3 of either tile are a
//                  lane's eight), so that w goes from the softmax to the product
//                  without leaving its lane; V^T comes from LDS by
//                  ds_read_b64_tr_b16 in the same order
// Sixteen-byte chunks of a V row are permuted by the row in pairs, which spreads
// the transposed reads over all banks (17 thousand conflicts in 17 million cycles
// of LDS).
//
// Up to 16 rows (few): memory is the bound.  K's operands come straight from
// memory to registers, V's rows to LDS that each wave has to itself; waves take the
// places of a step in turn and meet only at the end of a tile's run.  64 sequences of
// one token over up to 8192 places each: 197 us, 5.1 TB/s of 1.01 GB.  With four
// waves and twice the workgroups 224.
//
// More rows: a wave with rows of its own needs all of K and V, so eight waves share
// tiles of them in LDS (reading them from memory for each wave: 567 us for the tree
// below, now 172).  A tree of 64 tokens over 131072 places, 256 rows to a key head:
// 172 us, 3.1 TB/s and 0.80 PFLOP/s at once.  Two waves a SIMD, which the registers
// allow, keep the matrix cores 40% busy: what is not overlapped is the softmax's
// instructions between the two products.  (Wave priorities around the products, and
// the scores of two blocks before their softmax: no faster.)
//
// One token over few places is a chain of latencies (starts and lengths, pages, then K
// and V of a block for each of the waves, three turns of them over 700 places, the waves'
// sums): 17 us over 700 places, 10 over 16.
//
// Work is cut by df11_attention_plan.h; a tile that one workgroup does alone is
// written at once, the parts of the others go to the workspace and a second
// kernel joins them in order (5 to 12 us, 21 where prompts cut most tiles).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include <stdint.h>

#include "df11.h"
#include "df11_attention_plan.h"
#include "df11_device.h"
#include "df11_kv.h"
#include "df11_types.h"

namespace {

using df11::kFewStep;
using df11::kManyStep;
using df11::SeqShape;

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef short shortx4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kBlock = 32;   // places of one block of scores
// Waves of the kernel for few rows, by the head's padded size: as many as have room
// for their rows of V.
template <int KK>
constexpr uint32_t kFewWaves = KK > 4 ? 4 : 8;
static_assert(kFewStep == kFewWaves<4> * kBlock, "a step is a block for each wave");

// Parts of a tile whose loads one thread of the second kernel has in flight, and
// the most tiles that it joins.
constexpr uint32_t kJoinAtOnce = 8, kMaxCuts = 1024;

// A tile that a run begins and leaves to the runs after it.
struct Cut {
    int32_t begin;          // of its sequence: the first token, tokens
    uint32_t rows, head, tile;
    uint32_t run, last;     // runs that have parts of it; last 0: there is none
    uint32_t slot;          // of run's two slots; the others have it in their first
    uint32_t reserved;
};

struct AttentionArgs {
    df11::KvBatch b;
    df11::KvPages k, v;
    const void *q;
    void *out;
    float *lse;
    const uint8_t *mask;
    uint64_t q_stride, q_head_stride, out_stride, out_head_stride, mask_stride;
    uint64_t capacity;    // places of a sequence's pages
    float *parts;         // [workgroup][2][row][dim]
    float *stats;         // [workgroup][2][row][4]: reference times c, sums of the rounded weights and of them unrounded
    Cut *cut;             // [workgroup]; null where no tile is ever cut
    uint32_t page_magic, page_shift;  // df11::page_of
    float c;              // scale log2(e)
    uint32_t mask_cols, n_pages, page_size, kv_heads, group, dim, workgroups, tile_rows;
    uint32_t step, extra;  // places of a unit, units of a tile beside them
};

__device__ __forceinline__ floatx4 mfma(vec_t<bf16_t, 8> a, vec_t<bf16_t, 8> b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ floatx4 mfma(vec_t<fp16_t, 8> a, vec_t<fp16_t, 8> b, floatx4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Four operands of V^T: for each of four LDS addresses, 4 rows x 16 columns of
// 2-byte elements transposed across a quarter wave (lane i of the quarter passes
// the address of row i / 4, columns 4 (i mod 4) .. + 3, and receives column i of
// the four rows), and the same `next` bytes on.  (With the builtin for one read the
// compiler waits for every load to LDS in flight first; the block ends with its
// own wait, so that its results are there.)
template <int next>
__device__ __forceinline__ void read_transposed(const uint32_t (&at)[4], shortx4 (&x)[4][2]) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8\n\t"
        "ds_read_b64_tr_b16 %1, %8 offset:%12\n\t"
        "ds_read_b64_tr_b16 %2, %9\n\t"
        "ds_read_b64_tr_b16 %3, %9 offset:%12\n\t"
        "ds_read_b64_tr_b16 %4, %10\n\t"
        "ds_read_b64_tr_b16 %5, %10 offset:%12\n\t"
        "ds_read_b64_tr_b16 %6, %11\n\t"
        "ds_read_b64_tr_b16 %7, %11 offset:%12\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(x[0][0]), "=&v"(x[0][1]), "=&v"(x[1][0]), "=&v"(x[1][1]), "=&v"(x[2][0]), "=&v"(x[2][1]), "=&v"(x[3][0]),
          "=&v"(x[3][1])
        : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "n"(next));
}

// LDS address of a pointer into it.
__device__ __forceinline__ uint32_t lds_address(const uint8_t *p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const uint8_t *)p));
}

using Resource = __amdgpu_buffer_rsrc_t;

// Waits until at most VM vector memory loads and no LDS reads are in flight.  (The
// builtin and not assembly: the compiler then knows what has arrived, and adds no
// waits of its own that would drain the rest.)
template <int VM>
__device__ __forceinline__ void wait_loads() {
    static_assert(VM >= 0 && VM < 64, "six bits");
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4));
    asm volatile("" ::: "memory");
}

// 16 bytes a lane from `at` bytes on behind the wave-uniform address `from` to the
// wave-uniform LDS address dst + 16 lane.
__device__ __forceinline__ void load_rows_to_lds(const void *from, uint32_t at, uint8_t *dst) {
    const Resource r = __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(from), 0, 0xFFFFFFFFu, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void *)dst, 16, at, 0, 0, 0);
}

// The same from addresses of each lane's own.  (Slower than it looks: the
// compiler waits for every load in flight before it reads LDS after one of these,
// and not after the other kind.)
__device__ __forceinline__ void load_to_lds(const void *from, uint8_t *dst) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                     (__attribute__((address_space(3))) void *)dst, 16, 0, 0);
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// 2^(m - to), 0 for a reference of nothing.
__device__ __forceinline__ float weight_of(float m, float to) { return m == -INFINITY ? 0.0f : exp2_fast(m - to); }

// Whether a part adds nothing to its row.  (Scores that are all NaN leave no reference,
// but a sum that is NaN, which the row has to get.)
__device__ __forceinline__ bool adds_nothing(float weight, float sum) { return weight == 0.0f && sum == sum; }

__device__ __forceinline__ SeqShape shape_of(const AttentionArgs &a, uint32_t s) {
    return df11::seq_shape(a.b.starts[s], a.b.starts[s + 1], a.b.lengths[s], a.b.n_tokens, a.capacity, a.group,
                           a.tile_rows, a.step, a.extra, a.mask != nullptr);
}

// The sequence that holds a unit, and its first unit.
struct Found {
    uint32_t first, seq;
    SeqShape shape;
};

// Units of all sequences, by a whole workgroup of THREADS threads; a thread's own
// sequence of the first THREADS, and the units up to its end, in `mine`.
template <uint32_t THREADS>
__device__ __forceinline__ uint64_t scan_units(const AttentionArgs &a, uint32_t at, uint64_t base, SeqShape &shape,
                                               uint64_t &n, uint64_t &mine, uint64_t *s_part) {
    const uint32_t lane = threadIdx.x & 63u, wave = threadIdx.x / 64u, s = at + threadIdx.x;
    shape = shape_of(a, min(s, a.b.n_seqs - 1u));
    n = s < a.b.n_seqs ? df11::seq_units(shape, a.kv_heads) : 0;
    mine = n;
    const uint32_t here = min(64u, a.b.n_seqs - at);  // (lanes that have a sequence, in any wave)
    for (uint32_t m = 1; m < here; m <<= 1) {
        const uint64_t other = __shfl_up(mine, m);
        if (lane >= m) mine += other;
    }
    if (lane == here - 1u) s_part[wave] = mine;
    __syncthreads();
    uint64_t all = 0;
#pragma unroll
    for (uint32_t w = 0; w < THREADS / 64u; ++w) {
        if (at + 64u * w >= a.b.n_seqs) break;
        if (w == wave) mine += base + all;
        all += s_part[w];
    }
    return base + all;
}

// One tile's part of a run.
struct Part {
    SeqShape s;
    uint32_t seq, head, tile;
    uint32_t step0, step1;  // steps of this run
    uint32_t plain, limit;  // places that every row of the tile sees, that some row may see
    bool whole;             // no other run has steps of this tile
};

// A row of a part's tile: its token among the sequence's and its query head.
__device__ __forceinline__ void row_of(const AttentionArgs &a, const Part &p, uint32_t row, uint32_t &token,
                                       uint32_t &head) {
    const uint32_t at = p.tile * a.tile_rows + row;
    token = at / a.group;
    head = p.head * a.group + at % a.group;
}

// Weights that a reference allows before it moves, and how far, in powers of two, it
// lies below the largest score.
template <typename T>
constexpr float kRoom = std::is_same_v<T, fp16_t> ? 32768.0f : 256.0f;
template <typename T>
constexpr float kLead = std::is_same_v<T, fp16_t> ? 7.0f : 0.0f;

// What a head's chunks past head_dim read.
__device__ const uint4 g_zeros = {0, 0, 0, 0};

// What a wave keeps of its rows: M tiles of 16 from row0 of the part's tile on,
// lane l having row l mod 16 of each.
template <typename T, int KK, int M>
struct Rows {
    static constexpr int DP = 32 * KK;      // head_dim padded
    static constexpr int kChunks = DP / 8;  // 16-byte chunks of a row of K or V
    static constexpr int kTilesD = DP / 16;
    using Vec = vec_t<T, 8>;

    const AttentionArgs &a;
    const Part &p;
    uint32_t row0, lane, quarter, l16;

    Vec q[M][KK];
    floatx4 o[M][kTilesD];
    // A lane's row: its reference times c; the sum of its weights as they were rounded,
    // from a product with ones (four times the same); and this lane's part of their sum
    // unrounded, which only lse needs.  The quotient takes the first: its roundings are
    // the numerator's, and cancel as far as values are alike.  (The product adds to it
    // as to the numerator, in 3% of a call's time for many rows and none for few; rounded
    // weights added one by one take 6 to 7%.)
    float ref[M], l[M];
    floatx4 total[M];

    __device__ __forceinline__ Rows(const AttentionArgs &args, const Part &part, uint32_t first_row)
        : a(args), p(part), row0(first_row), lane(threadIdx.x & 63u), quarter(lane >> 4), l16(lane & 15u) {
#pragma unroll
        for (int i = 0; i < M; ++i) {
            ref[i] = -INFINITY;
            l[i] = 0.0f;
            total[i] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int d = 0; d < kTilesD; ++d) o[i][d] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        }
    }

    // Token and query head of this lane's row of row tile i.  Rows past the sequence's
    // last one have that one's: it is of this tile, so that out may lie on q (another
    // tile's rows may have been written), and what it sees and scores moves no
    // reference that it does not move itself.  Their sums go nowhere.
    __device__ __forceinline__ void query_of(int i, uint32_t &token, uint32_t &head) const {
        const uint32_t at = min(p.tile * a.tile_rows + row0 + 16u * i + l16, p.s.rows * a.group - 1u);
        token = at / a.group;
        head = p.head * a.group + at % a.group;
    }

    // Sends for the queries.
    __device__ __forceinline__ void load_queries() {
        const uint32_t last_chunk = a.dim / 8u - 1u;
#pragma unroll
        for (int i = 0; i < M; ++i) {
            uint32_t token, head;
            query_of(i, token, head);
            const T *row = static_cast<const T *>(a.q) + (static_cast<uint64_t>(p.s.begin) + token) * a.q_stride +
                           head * a.q_head_stride;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
                q[i][kk] = *reinterpret_cast<const Vec *>(row + 8u * min(4u * kk + quarter, last_chunk));
        }
    }

    // Zeros in their chunks past head_dim, as in K's.
    __device__ __forceinline__ void pad_queries() {
        if (a.dim == DP) return;
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int kk = 0; kk < KK; ++kk)
                if (4u * kk + quarter >= a.dim / 8u) q[i][kk] = Vec{};
    }

    // A pair of chunks of a row of V in LDS is kept at its number XOR this.
    static __device__ __forceinline__ uint32_t turn(uint32_t row) {
        return DP >= 128 ? row & 7u : (row >> 1) & 3u;
    }

    // The places of the block at key0 that a row sees, as far as this lane has
    // them: bit 4 t + e is place 16 t + 4 quarter + e.  (Bits and selects only:
    // out of nested branches around single elements of the scores the compiler
    // has made code that keeps the masked ones.)
    __device__ __forceinline__ uint32_t seen(uint32_t token, const uint8_t *mask_row, uint32_t key0, uint32_t valid) const {
        uint32_t bits = 0;
        if (mask_row && a.mask_cols) {
            // (eight loads at once, of the last column where there is none)
            uint32_t byte[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                byte[e] = mask_row[min(key0 + 16u * (e / 4) + 4u * quarter + e % 4 - p.s.length, a.mask_cols - 1u)];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                // (a cached place's j wraps)
                const uint32_t key = key0 + 16u * (e / 4) + 4u * quarter + e % 4, j = key - p.s.length;
                bits |= (key < p.s.length ? 1u : j < a.mask_cols && byte[e] ? 1u : 0u) << e;
            }
        } else {
            const uint32_t end = p.s.length + (mask_row ? 0u : token + 1u);  // places that the row sees
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint32_t key = key0 + 16u * t + 4u * quarter, n = key < end ? min(end - key, 4u) : 0u;
                bits |= ((1u << n) - 1u) << (4 * t);
            }
        }
        return bits & (((valid >> (4u * quarter)) & 15u) | (((valid >> (16u + 4u * quarter)) & 15u) << 4));
    }

    // The same of every row tile.
    __device__ __forceinline__ void look(uint32_t (&bits)[M], uint32_t key0, uint32_t valid) const {
#pragma unroll
        for (int i = 0; i < M; ++i) {
            uint32_t token, head;
            query_of(i, token, head);
            const uint8_t *mask_row = a.mask ? a.mask + (p.s.begin + static_cast<uint64_t>(token)) * a.mask_stride : nullptr;
            bits[i] = seen(token, mask_row, key0, valid);
        }
    }

    // Scores to weights (in s, and rounded in w).  A weight past the room (infinite
    // while there is no reference) says that the reference has to move: then
    // they are taken again, from the new one.  What a fused product keeps of a score
    // times c beside the reference, which was rounded, is the same for places of one
    // score in all blocks; but of references from 2^24 on it is more than a power of two
    // (from 2^31 on it makes the largest score's weight infinite): there, where scores
    // no longer tell places apart, weights are taken from products rounded alike.
    __device__ __forceinline__ void weigh(floatx4 (&s)[M][2], Vec (&w)[M]) {
        const T one = static_cast<T>(1.0f);
        floatx4 x[M][2];
        bool moves = false;
#pragma unroll
        for (int i = 0; i < M; ++i) {
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i][t][e] = exp2_fast(__builtin_fmaf(s[i][t][e], a.c, -ref[i]));
            // (all NaN: no reference, and nothing seen)
            moves |= !(largest(x[i]) <= kRoom<T>);
        }
        if (__ballot(moves)) {
#pragma clang fp contract(off)
#pragma unroll
            for (int i = 0; i < M; ++i) {
                float top = largest(s[i]);
                top = fmaxf(top, __shfl_xor(top, 16));
                const float to = fmaxf(ref[i], fmaxf(top, __shfl_xor(top, 32)) * a.c - kLead<T>);
                const float f = weight_of(ref[i], to);
                const float base = to == -INFINITY ? 0.0f : to;
                const bool far = !(fabsf(base) < 16777216.0f);
                ref[i] = to;
                l[i] *= f;
                total[i] *= f;
#pragma unroll
                for (int d = 0; d < kTilesD; ++d) o[i][d] *= f;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float rounded = s[i][t][e] * a.c - base;
                        x[i][t][e] = exp2_fast(far ? rounded : __builtin_fmaf(s[i][t][e], a.c, -base));
                    }
            }
        }
#pragma unroll
        for (int i = 0; i < M; ++i) {
            if (a.lse)
                l[i] += ((x[i][0][0] + x[i][0][1]) + (x[i][0][2] + x[i][0][3])) +
                        ((x[i][1][0] + x[i][1][1]) + (x[i][1][2] + x[i][1][3]));
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[i][t][e] = x[i][t][e];
                    w[i][4 * t + e] = static_cast<T>(x[i][t][e]);
                }
            total[i] = mfma(Vec{one, one, one, one, one, one, one, one}, w[i], total[i]);
        }
    }

    static __device__ __forceinline__ float largest(const floatx4 (&x)[2]) {
        return fmaxf(fmaxf(fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[0][2], x[0][3])), fmaxf(x[1][0], x[1][1])),
                     fmaxf(x[1][2], x[1][3]));
    }

    // A block's scores to o, where every row sees all of its places.
    __device__ __forceinline__ void take(floatx4 (&s)[M][2], const uint8_t *v) {
        Vec w[M];
        weigh(s, w);
        add(w, v);
    }

    // The same where rows may not.
    __device__ __forceinline__ void take_masked(floatx4 (&s)[M][2], const uint32_t (&bits)[M], const uint8_t *v) {
        bool some = false;
#pragma unroll
        for (int i = 0; i < M; ++i) {
            some |= bits[i] != 255u;
#pragma unroll
            for (int e = 0; e < 8; ++e) s[i][e / 4][e % 4] = (bits[i] >> e) & 1u ? s[i][e / 4][e % 4] : -INFINITY;
        }
        Vec w[M];
        weigh(s, w);
        if (__ballot(some) && bad_values(v)) {
            add_one_by_one(s, v);
        } else {
            add(w, v);
        }
    }

    // The block's part of o, its rows of V in LDS at v.
    __device__ __forceinline__ void add(const Vec (&w)[M], const uint8_t *v) {
        // (v is a multiple of 1 KB and a row of 32 bytes times a power of two, so that
        // d XOR the row's turn is one XOR of the address)
        const uint32_t row = 4u * quarter + (l16 >> 2);
        const uint32_t base = lds_address(v) + row * (2 * DP) + 32u * turn(row) + 8u * (l16 & 3u);
#pragma unroll
        for (int d = 0; d < kTilesD; d += 4) {
            const uint32_t at[4] = {base ^ (32u * d), base ^ (32u * (d + 1)), base ^ (32u * (d + 2)), base ^ (32u * (d + 3))};
            union {
                shortx4 s[4][2];
                Vec v[4];
            } u;
            read_transposed<16 * 2 * DP>(at, u.s);  // (16 rows on: the same turn)
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < M; ++i) o[i][d + e] = mfma(u.v[e], w[i], o[i][d + e]);
        }
    }

    // Whether the block's rows of V hold an infinity or a NaN: a product would
    // carry it to rows that do not see its place (0 * inf).
    __device__ __forceinline__ bool bad_values(const uint8_t *v) const {
        constexpr uint32_t kExponent = std::is_same_v<T, bf16_t> ? 0x7F80u : 0x7C00u;
        bool bad = false;
        for (int i = 0; i < static_cast<int>(kBlock) * DP * 2 / 1024; ++i) {
            const uint4 x = *reinterpret_cast<const uint4 *>(v + 1024 * i + 16 * lane);
            const uint32_t words[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                bad = bad || (words[e] & kExponent) == kExponent || ((words[e] >> 16) & kExponent) == kExponent;
        }
        return __ballot(bad) != 0;
    }

    // The same as add() without the matrix cores: places that a row does not see
    // are left out.
    __device__ __forceinline__ void add_one_by_one(const floatx4 (&s)[M][2], const uint8_t *v) {
#pragma unroll 1
        for (uint32_t row = 0; row < kBlock; ++row) {
            const uint32_t at = 4u * (row >> 4) + (row & 3u), from = l16 + 16u * ((row >> 2) & 3u);
            const T *at_v = reinterpret_cast<const T *>(v + row * (2 * DP)) + 4u * quarter;
#pragma unroll
            for (int i = 0; i < M; ++i) {
                float x = s[i][0][0];
#pragma unroll
                for (uint32_t e = 1; e < 8; ++e) x = at == e ? s[i][e / 4][e % 4] : x;
                x = static_cast<float>(static_cast<T>(__shfl(x, from)));
#pragma unroll
                for (int d = 0; d < kTilesD; ++d)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float y = static_cast<float>(at_v[16u * (d ^ turn(row)) + e]);
                        o[i][d][e] += x == 0.0f ? 0.0f : x * y;
                    }
            }
        }
    }
};

// A wave of the kernel for few rows: it has all the tile's rows, and the waves take
// the blocks of places in turn.
template <typename T, int KK, bool kWhole>
struct FewWave : Rows<T, KK, 1> {
    static constexpr int M = 1;
    static constexpr uint32_t kStep = kFewWaves<KK> * kBlock;  // places of all waves' turns
    using R = Rows<T, KK, M>;
    using Vec = typename R::Vec;
    using R::a, R::p, R::lane, R::quarter, R::l16, R::DP, R::kChunks;
    static constexpr int kVBytes = kBlock * DP * 2;
    static constexpr int kVLoads = kVBytes / 1024;
    static constexpr int kVRows = 64 / kChunks;  // rows of one load

    uint8_t *lds;  // two buffers of kVBytes
    const int32_t *table;
    Vec k[2][KK];
    uint32_t valid;  // of the block in k: places whose page exists

    __device__ __forceinline__ FewWave(const AttentionArgs &args, const Part &part, uint8_t *buffers)
        : R(args, part, 0u), lds(buffers), table(args.b.page_table + part.seq * args.b.table_stride) {}

    __device__ __forceinline__ uint32_t page_of(uint32_t place) const {
        return df11::page_of(place, a.page_magic, a.page_shift);
    }

    // Page of the place that lane l mod 32 has of the block at key0, or of the
    // last one.  (Nothing here uses what is loaded, which would wait for it.)
    __device__ __forceinline__ uint32_t load_id(uint32_t key0) const {
        return static_cast<uint32_t>(table[page_of(min(key0 + (lane & 31u), p.limit - 1u))]);
    }

    // Sends for the block at key0, or past the last one for rows that are not used
    // (the number of loads in flight is the same on every path): K to `to`, V to
    // the LDS buffer dst.
    __device__ __forceinline__ void issue(uint32_t key0, uint32_t id, Vec (&to)[2][KK], uint8_t *dst,
                                          uint32_t &valid_to) const {
        const bool there = id < a.n_pages && key0 + (lane & 31u) < p.limit;
        valid_to = static_cast<uint32_t>(__ballot(there));
        id = there ? id : 0u;
        // (a block of nothing reads one place over and over: 17.5 us against 18.1 for
        // one token over 700 places)
        const uint64_t k_stride = valid_to ? a.k.place_stride : 0, v_stride = valid_to ? a.v.place_stride : 0;
        const uint32_t last_chunk = a.dim / 8u - 1u;
        const T *kp = static_cast<const T *>(a.k.p) + p.head * a.k.head_stride;
        const T *vp = static_cast<const T *>(a.v.p) + p.head * a.v.head_stride;
        const uint32_t v_row = lane / kChunks, slot = lane % kChunks;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const T *row;
            if constexpr (kWhole) {
                const uint32_t key = key0 + 16u * t, page = __builtin_amdgcn_readlane(id, 16 * t);
                const uint32_t off = key - page_of(key) * a.page_size;
                row = kp + page * a.k.page_stride + off * k_stride + l16 * k_stride;
            } else {
                const uint32_t key = key0 + 16u * t + l16, page = __shfl(id, 16 * t + l16);
                const uint32_t off = key - page_of(key) * a.page_size;
                row = kp + page * a.k.page_stride + off * k_stride;
            }
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const uint32_t chunk = 4u * kk + quarter;
                to[t][kk] = *(chunk <= last_chunk ? reinterpret_cast<const Vec *>(row + 8u * chunk)
                                                  : reinterpret_cast<const Vec *>(&g_zeros));
            }
        }
#pragma unroll
        for (int i = 0; i < kVLoads; ++i) {
            const uint32_t r = i * kVRows + v_row;  // row of the block
            const uint32_t chunk = min(slot ^ (2u * R::turn(r)), last_chunk);
            if constexpr (kWhole) {
                const uint32_t t = i * kVRows / 16, key = key0 + 16u * t, page = __builtin_amdgcn_readlane(id, 16 * t);
                const uint32_t off = key - page_of(key) * a.page_size;
                load_rows_to_lds(vp + page * a.v.page_stride + off * v_stride,
                                 2u * ((r - 16u * t) * static_cast<uint32_t>(v_stride) + 8u * chunk), dst + 1024 * i);
            } else {
                const uint32_t key = key0 + r, page = __shfl(id, r);
                load_to_lds(vp + page * a.v.page_stride + (key - page_of(key) * a.page_size) * v_stride + 8u * chunk,
                            dst + 1024 * i);
            }
        }
    }

    __device__ __forceinline__ void scores(floatx4 (&s)[M][2]) const {
#pragma unroll
        for (int i = 0; i < M; ++i)
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                s[i][t] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) s[i][t] = mfma(k[t][kk], R::q[i][kk], s[i][t]);
            }
    }

    // Blocks from key0 on while they are seen whole, or all (kMasked).
    template <bool kMasked>
    __device__ __forceinline__ void blocks(uint32_t &key0, uint32_t end, uint32_t &id, uint8_t *&cur, uint8_t *&other) {
        while (key0 < end && (kMasked || (key0 + kBlock <= p.plain && valid == ~0u))) {
            // This block has landed, and the other buffer's last reads are back.
            wait_loads<0>();
            Vec next[2][KK];
            uint32_t next_valid = 0;
            const uint32_t then = load_id(key0 + 2u * kStep);
            issue(key0 + kStep, id, next, other, next_valid);
            id = then;
            floatx4 s[M][2];
            uint32_t bits[M];
            if constexpr (kMasked) R::look(bits, key0, valid);
            scores(s);
            if constexpr (kMasked) {
                R::take_masked(s, bits, cur);
            } else {
                R::take(s, cur);
            }
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int kk = 0; kk < KK; ++kk) k[t][kk] = next[t][kk];
            valid = next_valid;
            uint8_t *x = cur;
            cur = other;
            other = x;
            key0 += kStep;
        }
    }

    __device__ __forceinline__ void run(uint32_t wave) {
        uint32_t key0 = p.step0 * a.step + wave * kBlock;
        const uint32_t end = min(p.limit, p.step1 * a.step);
        if (key0 >= end) return;
        uint8_t *cur = lds, *other = lds + kVBytes;
        // (this wave's reads of the buffers, for the tile before, are back)
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        const uint32_t id0 = load_id(key0);
        uint32_t id = load_id(key0 + kStep);
        R::load_queries();
        issue(key0, id0, k, cur, valid);
        R::pad_queries();
        blocks<false>(key0, end, id, cur, other);
        blocks<true>(key0, end, id, cur, other);
        wait_loads<0>();  // (the buffers are used otherwise next)
    }
};

// A wave of the kernel for many rows: WR waves have the tile's rows, M row tiles
// each, and share the places that WK groups of waves take in turn.  K and V come
// to LDS in tiles of kTile places, in a ring of three: the tile after the next is
// sent for once every wave has left the one before this, at the one barrier of
// a tile.
template <typename T, int KK, int M, int WR, int WK, bool kWhole>
struct ManyWave : Rows<T, KK, M> {
    using R = Rows<T, KK, M>;
    using Vec = typename R::Vec;
    using R::a, R::p, R::lane, R::quarter, R::l16, R::DP, R::kChunks;
    static constexpr int kWaves = WR * WK;
    static constexpr int kTile = DP > 128 ? 32 : 64;
    static constexpr int kBlocks = kTile / static_cast<int>(kBlock) / WK;  // of a wave, a tile
    static_assert(kBlocks >= 1, "a group of waves has a block of a tile");
    static constexpr int kHalf = kTile * DP * 2;  // bytes of K or of V
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kLoads = kHalf / 1024 / kWaves;  // of a wave
    static_assert(kLoads * 1024 * kWaves == kHalf, "whole loads");
    static constexpr int kLoadRows = 64 / kChunks;

    uint32_t wave, group;
    uint8_t *lds;
    const int32_t *table;

    __device__ __forceinline__ ManyWave(const AttentionArgs &args, const Part &part, uint32_t w, uint8_t *ring)
        : R(args, part, (w % WR) * 16u * M), wave(w), group(w / WR), lds(ring),
          table(args.b.page_table + part.seq * args.b.table_stride) {}

    __device__ __forceinline__ uint32_t page_of(uint32_t place) const {
        return df11::page_of(place, a.page_magic, a.page_shift);
    }

    // Page of the place that lane l has of the tile at key0, or of the last one.
    // (Nothing here uses what is loaded, which would wait for it.)
    __device__ __forceinline__ uint32_t load_id(uint32_t key0) const {
        return static_cast<uint32_t>(table[page_of(min(key0 + lane % kTile, p.limit - 1u))]);
    }

    // Sends for the tile at key0, or past the last one for rows that are not used:
    // the number of loads in flight is the same on every path.
    __device__ __forceinline__ void issue(uint32_t key0, uint32_t id, uint8_t *stage, uint64_t &valid) const {
        const bool there = id < a.n_pages && key0 + lane % kTile < p.limit;
        valid = __ballot(there);
        id = there ? id : 0u;
        const uint32_t last_chunk = a.dim / 8u - 1u, slot = lane % kChunks;
        const T *kp = static_cast<const T *>(a.k.p) + p.head * a.k.head_stride;
        const T *vp = static_cast<const T *>(a.v.p) + p.head * a.v.head_stride;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const uint32_t load = wave + kWaves * i, r0 = load * kLoadRows, r = r0 + lane / kChunks;  // row of the tile
            const uint32_t k_chunk = slot ^ k_turn(r), v_chunk = slot ^ (2u * R::turn(r));
            uint8_t *k_to = stage + 1024u * load, *v_to = k_to + kHalf;
            if constexpr (kWhole) {
                const uint32_t key = key0 + r0, off = key - page_of(key) * a.page_size;
                const uint64_t page = __builtin_amdgcn_readlane(id, r0);
                const T *k_row = kp + page * a.k.page_stride + off * a.k.place_stride;
                const T *v_row = vp + page * a.v.page_stride + off * a.v.place_stride;
                const uint32_t row = lane / kChunks;
                load_rows_to_lds(k_row, 2u * (row * static_cast<uint32_t>(a.k.place_stride) + 8u * k_chunk), k_to);
                load_rows_to_lds(v_row, 2u * (row * static_cast<uint32_t>(a.v.place_stride) + 8u * v_chunk), v_to);
            } else {
                const uint32_t key = key0 + r, off = key - page_of(key) * a.page_size;
                const uint64_t page = __shfl(id, r);
                if (k_chunk <= last_chunk)
                    load_to_lds(kp + page * a.k.page_stride + off * a.k.place_stride + 8u * k_chunk, k_to);
                if (v_chunk <= last_chunk)
                    load_to_lds(vp + page * a.v.page_stride + off * a.v.place_stride + 8u * v_chunk, v_to);
            }
        }
    }

    // A chunk of a row of K in LDS is kept at its number XOR this.
    static __device__ __forceinline__ uint32_t k_turn(uint32_t row) { return row & (kChunks < 16 ? 7u : 15u); }

    __device__ __forceinline__ void scores(floatx4 (&s)[M][2], const uint8_t *k) const {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint8_t *row = k + (16u * t + l16) * (2 * DP);
#pragma unroll
            for (int i = 0; i < M; ++i) s[i][t] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
                const Vec f = *reinterpret_cast<const Vec *>(row + 16u * ((4u * kk + quarter) ^ k_turn(l16)));
#pragma unroll
                for (int i = 0; i < M; ++i) s[i][t] = mfma(f, R::q[i][kk], s[i][t]);
            }
        }
    }

    // Where a run stands: the tile at key0 is in cur, the next one in next or on its way.
    struct Ring {
        uint32_t key0, end, id;  // id: of the tile after the next
        uint64_t valid, valid_next;
        uint8_t *cur, *next, *free;
    };

    // Tiles from r.key0 on: kPlain while they are seen whole, kMasked all, kIdle all
    // for a wave without rows, which only sends for its part of them.
    enum Kind { kPlain, kMasked, kIdle };
    template <Kind kKind>
    __device__ __forceinline__ void tiles(Ring &r) {
        constexpr uint64_t kAll = kTile == 64 ? ~0ull : (1ull << (kTile % 64)) - 1u;
        while (r.key0 < r.end && (kKind != kPlain || (r.key0 + kTile <= p.plain && (r.valid & kAll) == kAll))) {
            // This tile has landed (the next one's loads, sent for after it, may be on
            // their way), and no wave reads the one before any more.
            wait_loads<2 * kLoads>();
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            uint64_t later = 0;
            // (the next id first: a wait for it leaves the tile's loads alone)
            const uint32_t then = load_id(r.key0 + 3u * kTile);
            issue(r.key0 + 2u * kTile, r.id, r.free, later);
            r.id = then;
            uint32_t bits[kBlocks][M];
            if constexpr (kKind == kMasked) {
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    const uint32_t at = (group * kBlocks + b) * kBlock;
                    R::look(bits[b], r.key0 + at, static_cast<uint32_t>(r.valid >> at));
                }
            }
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
                const uint32_t at = (group * kBlocks + b) * kBlock;
                const uint8_t *k = r.cur + at * (2 * DP), *v = k + kHalf;
                floatx4 s[M][2];
                if constexpr (kKind == kMasked) {
                    // (a wave's rows may end before the tile's places do)
                    bool some = false;
#pragma unroll
                    for (int i = 0; i < M; ++i) some |= bits[b][i] != 0;
                    if (__ballot(some)) {
                        scores(s, k);
                        R::take_masked(s, bits[b], v);
                    }
                } else if constexpr (kKind == kPlain) {
                    scores(s, k);
                    R::take(s, v);
                }
            }
            r.key0 += kTile;
            r.valid = r.valid_next;
            r.valid_next = later;
            uint8_t *x = r.cur;
            r.cur = r.next;
            r.next = r.free;
            r.free = x;
        }
    }

    // (called by all waves of the workgroup, with a barrier since the last use of the ring)
    __device__ __forceinline__ void run() {
        Ring r{p.step0 * a.step, min(p.limit, p.step1 * a.step), 0, 0, 0, lds, lds + kStage, lds + 2 * kStage};
        if (r.key0 >= r.end) return;
        if (!kWhole && a.dim != DP) {
            // Chunks past head_dim are never loaded: zeros, as in q.
            for (uint32_t at = threadIdx.x; at < 3u * kStage / 16u; at += 64u * kWaves)
                reinterpret_cast<uint4 *>(lds)[at] = uint4{0, 0, 0, 0};
            __syncthreads();
        }
        const uint32_t id0 = load_id(r.key0), id1 = load_id(r.key0 + kTile);
        r.id = load_id(r.key0 + 2u * kTile);
        R::load_queries();
        issue(r.key0, id0, r.cur, r.valid);
        issue(r.key0 + kTile, id1, r.next, r.valid_next);
        R::pad_queries();
        uint32_t token, head;
        row_of(a, p, R::row0, token, head);
        if (token < p.s.rows) {
            tiles<kPlain>(r);
            tiles<kMasked>(r);
        } else {
            tiles<kIdle>(r);
        }
        wait_loads<0>();  // (the ring is used otherwise next)
    }
};

// Joins the sums that WK groups of WR waves have of a part, row tile by row tile
// of each wave, and writes them: to out and lse if the part is whole, else to the
// workgroup's slot.
template <typename T, int KK, int M, int WR, int WK>
__device__ __forceinline__ void finish_part(const AttentionArgs &a, const Part &p, Rows<T, KK, M> &w, uint32_t wave,
                                            uint8_t *lds, float (*s_stats)[16][3], uint64_t slot) {
    constexpr int DP = 32 * KK, kStride = DP + 4;
    constexpr uint32_t kWaveFloats = 16 * kStride;
    float *sums = reinterpret_cast<float *>(lds);
#pragma unroll
    for (int i = 0; i < M; ++i) {
        float total = w.total[i][0], l = 0.0f;
        if (a.lse) {
            l = w.l[i] + __shfl_xor(w.l[i], 16);
            l += __shfl_xor(l, 32);
        }
        // (every wave's reads of the places, and of the row tile before, are back)
        __syncthreads();
        if (w.quarter == 0) {
            s_stats[wave][w.l16][0] = w.ref[i];
            s_stats[wave][w.l16][1] = total;
            s_stats[wave][w.l16][2] = l;
        }
#pragma unroll
        for (int d = 0; d < Rows<T, KK, M>::kTilesD; ++d)
            *reinterpret_cast<floatx4 *>(sums + wave * kWaveFloats + w.l16 * kStride + 16 * d + 4 * w.quarter) = w.o[i][d];
        __syncthreads();
        for (uint32_t at = threadIdx.x; at < WR * 16u * (DP / 8); at += 64u * WR * WK) {
            const uint32_t from = at / (DP / 8), d = 8u * (at % (DP / 8)), wr = from / 16u, r = from % 16u;
            const uint32_t row = (wr * M + i) * 16u + r;
            uint32_t token, head;
            row_of(a, p, row, token, head);
            if (token >= p.s.rows || d >= a.dim) continue;
            float top = -INFINITY, total = 0.0f, whole = 0.0f, sum[8] = {};
#pragma unroll
            for (uint32_t x = 0; x < WK; ++x) top = fmaxf(top, s_stats[x * WR + wr][r][0]);
#pragma unroll
            for (uint32_t x = 0; x < WK; ++x) {
                const uint32_t other = x * WR + wr;
                const float f = weight_of(s_stats[other][r][0], top);
                if (adds_nothing(f, s_stats[other][r][1])) continue;
                total += f * s_stats[other][r][1];
                whole += f * s_stats[other][r][2];
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += f * sums[other * kWaveFloats + r * kStride + d + e];
            }
            if (p.whole) {
                const uint64_t t = static_cast<uint64_t>(p.s.begin) + token;
                const float f = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] *= f;
                store_vec<T, 8>(static_cast<T *>(a.out) + t * a.out_stride + head * a.out_head_stride + d, sum);
                if (a.lse && d == 0)
                    a.lse[t * (a.kv_heads * a.group) + head] =
                        total == 0.0f ? -INFINITY : (top + log2f(whole)) * 0.69314718055994531f;
            } else {
                float *to = a.parts + (slot * a.tile_rows + row) * a.dim + d;
                store_vec<float, 4>(to, *reinterpret_cast<float(*)[4]>(&sum[0]));
                store_vec<float, 4>(to + 4, *reinterpret_cast<float(*)[4]>(&sum[4]));
                const float st[4] = {top, total, whole, 0.0f};
                if (d == 0) store_vec<float, 4>(a.stats + (slot * a.tile_rows + row) * 4u, st);
            }
        }
    }
    __syncthreads();
}

// A workgroup's run of units: f(part, slot) for every tile that it has a part of.
template <uint32_t THREADS, typename F>
__device__ __forceinline__ void for_each_part(const AttentionArgs &a, F f) {
    __shared__ uint64_t s_part[THREADS / 64];
    __shared__ Found s_found;
    // Units of all sequences; then the one that this run begins in.  (Up to THREADS
    // sequences the first round has both.)
    uint64_t units = 0, n = 0, mine = 0;
    SeqShape shape;
    for (uint32_t at = 0; at < a.b.n_seqs; at += THREADS) {
        if (at) __syncthreads();
        units = scan_units<THREADS>(a, at, units, shape, n, mine, s_part);
    }
    const bool none = units == 0 || units >= df11::kMaxUnits;
    const uint32_t all = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(units));
    const uint32_t runs = none ? 0u : df11::runs_of(all, a.workgroups);
    // What the second kernel finds of a run: the tile that it begins and leaves.
    if (a.cut && blockIdx.x >= runs && threadIdx.x == 0) a.cut[blockIdx.x].last = 0;
    if (blockIdx.x >= runs) return;
    const uint32_t run = df11::run_of_workgroup(blockIdx.x, runs);
    uint32_t u = df11::run_begin(run, all, runs);
    const uint32_t end = df11::run_begin(run + 1u, all, runs);
    uint64_t base = 0;
    for (uint32_t at = 0; at < a.b.n_seqs; at += THREADS) {
        if (a.b.n_seqs > THREADS) {
            __syncthreads();
            base = scan_units<THREADS>(a, at, base, shape, n, mine, s_part);
        }
        if (u >= mine - n && u < mine) s_found = Found{static_cast<uint32_t>(mine - n), at + threadIdx.x, shape};
    }
    __syncthreads();
    const uint32_t first = __builtin_amdgcn_readfirstlane(s_found.first);
    bool begun = true;  // the run's first tile may have begun in the run before
    bool left = false;
    Part p;
    p.s = s_found.shape;
    p.seq = __builtin_amdgcn_readfirstlane(s_found.seq);
    const uint32_t one = static_cast<uint32_t>(df11::units_before(p.s, p.s.tiles));  // of a key head
    p.head = (u - first) / one;
    p.tile = df11::tile_of(p.s, u - first - p.head * one);
    uint32_t tile_first = first + p.head * one + static_cast<uint32_t>(df11::units_before(p.s, p.tile));
    while (u < end) {
        const uint32_t tile_end = tile_first + df11::tile_units(p.s, p.tile), to = min(end, tile_end);
        p.step0 = df11::steps_before(p.s, u - tile_first);
        p.step1 = df11::steps_before(p.s, to - tile_first);
        u = to;
        if (p.step0 != p.step1) {
            p.plain = df11::tile_plain(p.s, p.tile, a.tile_rows, a.group, a.mask != nullptr);
            p.limit = df11::tile_places(p.s, p.tile, a.tile_rows, a.group, a.mask != nullptr);
            p.whole = p.step0 == 0 && to == tile_end;
            if (a.cut && p.step0 == 0 && !p.whole) {
                left = true;
                if (threadIdx.x == 0)
                    a.cut[run] = Cut{p.s.begin, p.s.rows, p.head, p.tile, run, df11::run_of(tile_end - 1u, all, runs),
                                     begun ? 0u : 1u, 0u};
            }
            f(p, 2ull * run + (begun ? 0u : 1u));
            begun = false;
        }
        // The next tile, of the next key head, of the next sequence that has one.
        tile_first = tile_end;
        if (++p.tile < p.s.tiles) continue;
        p.tile = 0;
        if (++p.head < a.kv_heads) continue;
        p.head = 0;
        if (u == end) break;
        do {
            if (++p.seq == a.b.n_seqs) {  // (never: units are left)
                u = end;
                break;
            }
            p.s = shape_of(a, p.seq);
        } while (!p.s.tiles);
    }
    if (a.cut && !left && threadIdx.x == 0) a.cut[run].last = 0;
}

// Up to 16 rows: the workgroup's waves have them all, and the places in turn.
template <typename T, int KK, bool kWhole>
__global__ __launch_bounds__(64 * kFewWaves<KK>) __attribute__((amdgpu_waves_per_eu(kFewWaves<KK> / 4)))
void df11_attention_few_kernel(AttentionArgs a) {
    using W = FewWave<T, KK, kWhole>;
    constexpr uint32_t kWaves = kFewWaves<KK>, kWaveBytes = 2u * W::kVBytes;
    static_assert(kWaveBytes >= 16 * (W::DP + 4) * 4, "a row tile's sums fit a wave's buffers");
    __shared__ __align__(1024) uint8_t s_mem[kWaves * kWaveBytes];
    __shared__ float s_stats[kWaves][16][3];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u);
    for_each_part<64 * kWaves>(a, [&](const Part &p, uint64_t slot) {
        W w(a, p, s_mem + wave * kWaveBytes);
        w.run(wave);
        finish_part<T, KK, 1, 1, kWaves>(a, p, w, wave, s_mem, s_stats, slot);
    });
}

// More rows: eight waves share tiles of places in LDS.
template <typename T, int KK, int M, int WR, int WK, bool kWhole>
__global__ __launch_bounds__(64 * WR * WK) __attribute__((amdgpu_waves_per_eu(WR * WK / 4)))
void df11_attention_many_kernel(AttentionArgs a) {
    using W = ManyWave<T, KK, M, WR, WK, kWhole>;
    constexpr uint32_t kSums = WR * WK * 16 * (W::DP + 4) * 4;
    __shared__ __align__(1024) uint8_t s_mem[3 * W::kStage > kSums ? 3 * W::kStage : kSums];
    __shared__ float s_stats[WR * WK][16][3];
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u);
    for_each_part<64 * WR * WK>(a, [&](const Part &p, uint64_t slot) {
        W w(a, p, wave, s_mem);
        w.run();
        finish_part<T, KK, M, WR, WK>(a, p, w, wave, s_mem, s_stats, slot);
    });
}

// Joins `at`-th vector of eight elements of a cut tile, row by row.  kWaves: waves of
// the workgroup that take the vector's parts together, a stretch each, in the
// order of the places.
template <typename T, uint32_t kWaves>
__device__ __forceinline__ void join_vector(const AttentionArgs &a, const Cut &c, uint32_t at, float (*s_sum)[11][64]) {
    const uint32_t chunks = a.dim / 8u, row = at / chunks, d = 8u * (at % chunks), lane = threadIdx.x & 63u;
    const uint32_t wave = kWaves > 1 ? threadIdx.x / 64u : 0u;
    const uint32_t in_tiles = c.tile * a.tile_rows + row, token = in_tiles / a.group;
    const bool there = row < a.tile_rows && token < c.rows;
    const uint32_t in = there ? row : 0u;
    const auto slot_of = [&](uint32_t r) { return (2ull * r + (r == c.run ? c.slot : 0u)) * a.tile_rows + in; };
    const uint32_t each = (c.last - c.run + kWaves) / kWaves;
    const uint32_t begin = c.run + wave * each, end = min(begin + each, c.last + 1u);
    float top = -INFINITY, total = 0.0f, whole = 0.0f, sum[8] = {};
    for (uint32_t r = begin; r < end; r += kJoinAtOnce) {
        float st[kJoinAtOnce][4], v[kJoinAtOnce][8];
#pragma unroll
        for (uint32_t k = 0; k < kJoinAtOnce; ++k) {  // (past the last one again, not added)
            const uint64_t slot = slot_of(min(r + k, end - 1u));
            load_vec<float, 4>(a.stats + slot * 4u, st[k]);
            load_vec<float, 4>(a.parts + slot * a.dim + d, *reinterpret_cast<float(*)[4]>(&v[k][0]));
            load_vec<float, 4>(a.parts + slot * a.dim + d + 4, *reinterpret_cast<float(*)[4]>(&v[k][4]));
        }
        float to = top;
#pragma unroll
        for (uint32_t k = 0; k < kJoinAtOnce; ++k) to = fmaxf(to, st[k][0]);
        const float old = weight_of(top, to);
        total *= old;
        whole *= old;
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] *= old;
#pragma unroll
        for (uint32_t k = 0; k < kJoinAtOnce; ++k) {
            const float f = weight_of(st[k][0], to);
            if (r + k >= end || adds_nothing(f, st[k][1])) continue;
            total += f * st[k][1];
            whole += f * st[k][2];
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += f * v[k][e];
        }
        top = to;
    }
    if constexpr (kWaves > 1) {
        __syncthreads();  // (the vectors before have been read)
        s_sum[wave][8][lane] = top;
        s_sum[wave][9][lane] = total;
        s_sum[wave][10][lane] = whole;
#pragma unroll
        for (int e = 0; e < 8; ++e) s_sum[wave][e][lane] = sum[e];
        __syncthreads();
        if (wave) return;
#pragma unroll
        for (uint32_t w = 1; w < kWaves; ++w) {
            const float to = fmaxf(top, s_sum[w][8][lane]), old = weight_of(top, to), f = weight_of(s_sum[w][8][lane], to);
            total *= old;
            whole *= old;
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] *= old;
            if (!adds_nothing(f, s_sum[w][9][lane])) {
                total += f * s_sum[w][9][lane];
                whole += f * s_sum[w][10][lane];
#pragma unroll
                for (int e = 0; e < 8; ++e) sum[e] += f * s_sum[w][e][lane];
            }
            top = to;
        }
    }
    if (!there) return;
    const float f = total == 0.0f ? 0.0f : 1.0f / total;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] *= f;
    const uint64_t t = static_cast<uint64_t>(c.begin) + token;
    const uint32_t head = c.head * a.group + in_tiles % a.group;
    store_vec<T, 8>(static_cast<T *>(a.out) + t * a.out_stride + head * a.out_head_stride + d, sum);
    if (a.lse && d == 0)
        a.lse[t * (a.kv_heads * a.group) + head] =
            total == 0.0f ? -INFINITY : (top + log2f(whole)) * 0.69314718055994531f;
}

// Joins the parts of the tiles that runs begin and leave to others.  Every
// workgroup finds all of them, in the same order, those of many parts first, and
// takes its share of their vectors: 64 at a time with all four waves, or of a tile
// of few parts 64 for each wave.
template <typename T>
__global__ __launch_bounds__(256) void df11_attention_join_kernel(AttentionArgs a) {
    __shared__ uint32_t s_count[2][4], s_cut[2][kMaxCuts];
    __shared__ float s_sum[4][11][64];
    const uint32_t lane = threadIdx.x & 63u, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64u);
    uint32_t found[2] = {0, 0};  // of many parts, of few
    for (uint32_t at = 0; at < a.workgroups; at += 256u) {
        const uint32_t w = at + threadIdx.x;
        uint32_t parts = 0;
        if (w < a.workgroups && a.cut[w].last) parts = a.cut[w].last - a.cut[w].run + 1u;
        const uint64_t of[2] = {__ballot(parts > kJoinAtOnce), __ballot(parts && parts <= kJoinAtOnce)};
        __syncthreads();
        if (lane < 2u) s_count[lane][wave] = static_cast<uint32_t>(__popcll(of[lane]));
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            uint32_t first = found[k];
#pragma unroll
            for (uint32_t x = 0; x < 4u; ++x) {
                if (x < wave) first += s_count[k][x];
                found[k] += s_count[k][x];
            }
            if ((of[k] >> lane) & 1u) s_cut[k][first + __popcll(of[k] & ((1ull << lane) - 1u))] = w;
        }
    }
    __syncthreads();
    const uint32_t items = (a.tile_rows * (a.dim / 8u) + 63u) / 64u;
    for (uint32_t i = blockIdx.x; i < found[0] * items; i += gridDim.x)
        join_vector<T, 4>(a, a.cut[s_cut[0][i / items]], (i % items) * 64u + lane, s_sum);
    for (uint32_t i = blockIdx.x * 4u + wave; i < found[1] * items; i += gridDim.x * 4u)
        join_vector<T, 1>(a, a.cut[s_cut[1][i / items]], (i % items) * 64u + lane, s_sum);
}

// The kernels, by the rows of their tiles.
template <typename T, int KK>
const void *pick_rows(uint32_t rows, bool whole) {
    if (rows == 16)
        return whole ? reinterpret_cast<const void *>(&df11_attention_few_kernel<T, KK, true>)
                     : reinterpret_cast<const void *>(&df11_attention_few_kernel<T, KK, false>);
    const auto many = [&](auto m, auto wr, auto wk) {
        constexpr int M = decltype(m)::value, WR = decltype(wr)::value, WK = decltype(wk)::value;
        return whole ? reinterpret_cast<const void *>(&df11_attention_many_kernel<T, KK, M, WR, WK, true>)
                     : reinterpret_cast<const void *>(&df11_attention_many_kernel<T, KK, M, WR, WK, false>);
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    const std::integral_constant<int, 4> four;
    const std::integral_constant<int, 8> eight;
    if constexpr (KK == 8) {
        return rows == 64 ? many(one, four, one) : many(one, eight, one);
    } else {
        return rows == 64 ? many(one, four, two) : rows == 128 ? many(two, four, two) : many(two, eight, one);
    }
}

// Rows of a tile: enough for the rows that a sequence has on average (the host
// knows no more than that).  Measured, eight sequences over 4096 places, heads of
// 128, tiles of 16 / 64 / 128 / 256 rows: 41.7 / 43.7 / 47.9 / 56.6 us at 16 rows,
// 47.3 / 44.4 / 48.1 / 57.2 at 20, 66.2 / 47.3 / 50.4 / 59.7 at 64, 118 / 66.2 / 52.1 /
// 59.4 at 68, 112 / 68.7 / 54.8 / 62.3 at 128, 197 / 92.5 / 72.6 / 67.8 at 132, 201 / 104 /
// 80.1 / 75.1 at 256, and 1059 / 371 / 260 / 221 at 2048 over 2048.  Heads of 64 and 256
// have the same order but for 20 rows of 64 (25.7 / 29.4).
uint32_t pick_tile(uint32_t dim, uint64_t rows) {
    return rows <= 16 ? 16 : rows <= 64 ? 64 : rows <= 128 || dim > 128 ? 128 : 256;
}

uint32_t tile_threads(uint32_t dim, uint32_t rows) { return dim > 128 && rows <= 64 ? 256 : 512; }

template <typename T>
const void *pick_kernel(uint32_t dim, uint32_t rows, bool whole) {
    return dim <= 64 ? pick_rows<T, 2>(rows, whole) : dim <= 128 ? pick_rows<T, 4>(rows, whole) : pick_rows<T, 8>(rows, whole);
}

// Largest stride between places whose 16 fit 32 bits of offset.
constexpr uint64_t kMaxPlaceStride = 1u << 26;

// How a call is launched.
struct Plan {
    const void *fn;
    uint32_t tile_rows, threads, workgroups, step, extra;
    uint64_t parts, stats, cut;  // bytes; 0 where no tile is ever cut
};

int make_plan(const df11_kv_cache &c, const df11_kv_batch &b, uint32_t q_heads, Plan &p) {
    int dev = 0, cus = 0;
    if (device_cus(dev, cus)) return DF11_E_HIP;
    const uint32_t group = q_heads / c.heads;
    const uint64_t rows = static_cast<uint64_t>((b.n_tokens + b.n_seqs - 1) / b.n_seqs) * group;
    p.tile_rows = pick_tile(c.head_dim, rows);
    p.threads = tile_threads(c.head_dim, p.tile_rows);
    // Whether the rows of one load are places of one page, and fill it: then a load
    // has one address and 32-bit offsets.
    const bool few = p.tile_rows == 16;
    const uint32_t together = few ? 16 : 8;
    const bool whole = c.page_size % together == 0 && (few || c.head_dim == 64 || c.head_dim == 128 || c.head_dim == 256) &&
                       c.k_place_stride <= kMaxPlaceStride && c.v_place_stride <= kMaxPlaceStride;
    p.fn = c.dtype == DF11_BF16 ? pick_kernel<bf16_t>(c.head_dim, p.tile_rows, whole)
                                : pick_kernel<fp16_t>(c.head_dim, p.tile_rows, whole);
    const int per_cu = resident_per_cu(p.fn, p.threads, dev, 0);
    if (per_cu < 1) return DF11_E_HIP;
    const uint64_t capacity = static_cast<uint64_t>(b.table_pages) * c.page_size;
    const uint64_t tiles = (static_cast<uint64_t>(b.n_tokens) * group + p.tile_rows - 1) / p.tile_rows + b.n_seqs;
    // (an upper bound of the tiles, at most twice as many)
    const uint32_t uncut = df11::whole_places(few, tiles * c.heads, static_cast<uint32_t>(cus), c.head_dim);
    p.step = df11::unit_places(capacity, few, uncut);
    // (a tile without a mask may count a unit for its own tokens beside the pages')
    p.extra = df11::extra_units(capacity, few, uncut, c.head_dim);
    const uint64_t units = tiles * c.heads * ((capacity + p.step - 1) / p.step + 2 + p.extra);
    if (static_cast<uint64_t>(b.n_tokens) * group >= (1ull << 31) || units >= df11::kMaxUnits) return DF11_E_TOO_LARGE;
    p.workgroups = static_cast<uint32_t>(std::min<uint64_t>({static_cast<uint64_t>(cus) * per_cu, units, kMaxCuts}));
    const uint64_t slots = capacity > p.step ? 2ull * p.workgroups * p.tile_rows : 0;
    p.parts = round_up(slots * c.head_dim * 4, 256);
    p.stats = round_up(slots * 16, 256);
    p.cut = slots ? round_up(p.workgroups * sizeof(Cut), 256) : 0;
    return DF11_OK;
}

df11_attention used_strides(df11_attention a, uint32_t n_tokens) {
    for (uint64_t *s : {&a.q_stride, &a.out_stride, &a.mask_stride}) *s = kv_stride(n_tokens, *s);
    for (uint64_t *s : {&a.q_head_stride, &a.out_head_stride}) *s = kv_stride(a.q_heads, *s);
    return a;
}

// Checks of what comes beside the cache and the batch (already checked); the
// spans of q and out in bytes.
int check_attention(const df11_kv_cache &c, const df11_kv_batch &b, const df11_attention *a, uint64_t &q_span,
                    uint64_t &out_span) {
    if (!a->q_heads || a->q_heads > kMaxKvHeads || a->q_heads % c.heads || !(a->scale > 0.0f) ||
        !std::isfinite(a->scale))
        return DF11_E_INVALID_ARG;
    if (b.n_tokens == 0 || b.n_seqs == 0) return DF11_OK;
    if (!a->q || !a->out || !aligned(a->q, 16) || !aligned(a->out, 16)) return DF11_E_INVALID_ARG;
    const uint64_t strides[] = {a->q_stride, a->q_head_stride, a->out_stride, a->out_head_stride};
    for (const uint64_t s : strides)
        if (s % 8 || s >= kMaxKvStride) return DF11_E_INVALID_ARG;
    if (!kv_apart(b.n_tokens, a->out_stride, a->q_heads, a->out_head_stride, c.head_dim)) return DF11_E_INVALID_ARG;
    if (a->lse && !aligned(a->lse, 4)) return DF11_E_INVALID_ARG;
    if (a->mask && a->mask_stride >= kMaxKvStride) return DF11_E_INVALID_ARG;
    q_span = 2 * kv_span(b.n_tokens, a->q_stride, a->q_heads, a->q_head_stride, c.head_dim);
    out_span = 2 * kv_span(b.n_tokens, a->out_stride, a->q_heads, a->out_head_stride, c.head_dim);
    return DF11_OK;
}

}  // namespace

extern "C" {

uint64_t df11_tree_attention_workspace(const df11_kv_cache *c, const df11_kv_batch *b, const df11_attention *given) {
    uint64_t k_span = 0, v_span = 0, q_span = 0, out_span = 0;
    Plan p{};
    if (check_kv(c, b, k_span, v_span) || !given) return 0;
    const df11_attention used = used_strides(*given, b->n_tokens), *a = &used;
    if (check_attention(*c, *b, a, q_span, out_span)) return 0;
    if (b->n_tokens == 0 || b->n_seqs == 0 || make_plan(*c, *b, a->q_heads, p)) return 0;
    return p.parts + p.stats + p.cut;
}

int df11_tree_attention(const df11_kv_cache *c, const df11_kv_batch *b, const df11_attention *given, void *workspace,
                        uint64_t workspace_bytes, void *hip_stream) {
    uint64_t k_span = 0, v_span = 0, q_span = 0, out_span = 0;
    int rc = check_kv(c, b, k_span, v_span);
    if (!rc && !given) rc = DF11_E_INVALID_ARG;
    if (rc) return rc;
    const df11_attention used = used_strides(*given, b->n_tokens), *a = &used;
    rc = check_attention(*c, *b, a, q_span, out_span);
    if (rc || b->n_tokens == 0 || b->n_seqs == 0) return rc;
    // Outputs stay clear of everything that is read, but out may lie exactly on q, or
    // beside it in the rows of one tensor.
    const uint64_t lse_span = a->lse ? 4ull * b->n_tokens * a->q_heads : 0;
    const uint64_t mask_span = a->mask && a->mask_cols ? (b->n_tokens - 1ull) * a->mask_stride + a->mask_cols : 0;
    const bool on_q = a->q == a->out && a->q_stride == a->out_stride && a->q_head_stride == a->out_head_stride;
    const auto runs = [&](const void *p, uint64_t stride, uint64_t head_stride) {
        return runs_of(p, 2ull * c->head_dim, {{b->n_tokens, 2 * stride}, {a->q_heads, 2 * head_stride}});
    };
    const bool off_q = lie_apart(runs(a->out, a->out_stride, a->out_head_stride), runs(a->q, a->q_stride, a->q_head_stride));
    const void *outs[] = {a->out, a->lse, workspace};
    uint64_t spans[] = {out_span, lse_span, 0};
    const auto clear = [&](int i) {
        for (int j = 0; j < i; ++j)
            if (overlaps(outs[i], spans[i], outs[j], spans[j])) return false;
        return !overlaps(outs[i], spans[i], c->k, k_span) && !overlaps(outs[i], spans[i], c->v, v_span) &&
               (i == 0 ? on_q || off_q : !overlaps(outs[i], spans[i], a->q, q_span)) &&
               !overlaps(outs[i], spans[i], a->mask, mask_span) && clear_of_batch(*b, outs[i], spans[i]);
    };
    if (!clear(0) || !clear(1)) return DF11_E_INVALID_ARG;
    Plan p{};
    rc = make_plan(*c, *b, a->q_heads, p);
    if (rc) return rc;
    spans[2] = p.parts + p.stats + p.cut;
    if (spans[2] && (!workspace || !aligned(workspace, 256))) return DF11_E_INVALID_ARG;
    if (workspace_bytes < spans[2]) return DF11_E_BUFFER_TOO_SMALL;
    if (!clear(2)) return DF11_E_INVALID_ARG;
    AttentionArgs k{};
    k.b = kernel_batch(*b);
    k.k = kernel_pages(c->k, c->k_page_stride, c->k_place_stride, c->k_head_stride, *c);
    k.v = kernel_pages(c->v, c->v_page_stride, c->v_place_stride, c->v_head_stride, *c);
    k.q = a->q;
    k.out = a->out;
    k.lse = a->lse;
    k.mask = a->mask;
    k.q_stride = a->q_stride;
    k.q_head_stride = a->q_head_stride;
    k.out_stride = a->out_stride;
    k.out_head_stride = a->out_head_stride;
    k.mask_stride = a->mask_stride;
    k.capacity = static_cast<uint64_t>(b->table_pages) * c->page_size;
    k.parts = static_cast<float *>(workspace);
    k.stats = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + p.parts);
    k.cut = p.cut ? reinterpret_cast<Cut *>(static_cast<uint8_t *>(workspace) + p.parts + p.stats) : nullptr;
    k.page_shift = df11::page_shift(c->page_size);
    k.page_magic = df11::page_magic(c->page_size, k.page_shift);
    k.c = a->scale * 1.44269504088896341f;
    k.mask_cols = a->mask_cols;
    k.n_pages = c->n_pages;
    k.page_size = c->page_size;
    k.kv_heads = c->heads;
    k.group = a->q_heads / c->heads;
    k.dim = c->head_dim;
    k.workgroups = p.workgroups;
    k.tile_rows = p.tile_rows;
    k.step = p.step;
    k.extra = p.extra;
    (void)hipGetLastError();
    const hipStream_t stream = static_cast<hipStream_t>(hip_stream);
    void *params[] = {&k};
    rc = launch_kernel(p.fn, dim3(p.workgroups), dim3(p.threads), params, 0, stream, nullptr, nullptr);
    if (rc || !spans[2]) return rc;
    const void *join = c->dtype == DF11_BF16 ? reinterpret_cast<const void *>(&df11_attention_join_kernel<bf16_t>)
                                             : reinterpret_cast<const void *>(&df11_attention_join_kernel<fp16_t>);
    // (every item its own workgroup where that fills the chip no more than twice)
    const uint64_t items = static_cast<uint64_t>(p.workgroups) * ((p.tile_rows * (c->head_dim / 8) + 63) / 64);
    return launch_kernel(join, dim3(static_cast<uint32_t>(std::min<uint64_t>(items, 2ull * kMaxCuts))), dim3(256), params, 0,
                         stream, nullptr, nullptr);
}

}  // extern "C"
