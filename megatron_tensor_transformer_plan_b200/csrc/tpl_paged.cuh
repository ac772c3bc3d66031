// What the paged-cache kernels share: the view of a ragged batch over the
// pages, with the bounds checks of everything the device arrays say (a page
// id, length or start outside its range is recorded in the error word and
// replaced by one that is in bounds), and the append.
#pragma once

#include <cuda_bf16.h>

#include "tpl_common.cuh"
#include "tpl_internal.h"
#include "tpl_paged_ws.h"

namespace tpl {

// A kernel that needs nothing of the one before it, but of those before that, may start
// without waiting.  Starting says nothing about memory: what it may read is passed on by
// this word, which the kernel between sets after its own wait (its wait made the earlier
// results visible to it, the release store passes them on to whoever acquires the word).
// A reader that does not see it set waits instead.  A later kernel of the call, which has
// waited for the reader, clears it.
__device__ __forceinline__ void pdl_pass_on(unsigned *word) {
    asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(word), "r"(1u) : "memory");
}
__device__ __forceinline__ bool pdl_passed_on(const unsigned *word) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(word) : "memory");
    // (the copy engine's reads too)
    asm volatile("fence.proxy.async.global;" ::: "memory");
    return v == 1u;
}

constexpr unsigned kErrPaged = 32u;  // error word: a page id, length or start out of range

struct PagedView {
    const int32_t *table;     // [n_seqs][max_pages], rows table_stride apart
    int64_t table_stride;
    const int32_t *kv_len;    // [n_seqs]
    const int32_t *q_start;   // [n_seqs + 1], or NULL: one token per sequence
    int32_t max_pages, n_pages, page_shift, n_seqs, n_tokens, nkv, nkv_s;
};

// The work of a launch, U units, is cut into G equal ranges, one per CTA: the
// first unit of range c, and the range that unit x lies in (the last c with
// U c / G <= x).  Divisions of 64 bits take some hundred cycles, those of 32 a
// few tens, and most launches are small.
__device__ __forceinline__ int64_t paged_div(int64_t a, int64_t b) {
    return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}
__device__ __forceinline__ int64_t paged_cut(int64_t U, int G, int c) { return paged_div(U * c, G); }
__device__ __forceinline__ int paged_cta_of(int64_t U, int G, int64_t x) { return (int)paged_div((x + 1) * G - 1, U); }

__device__ __forceinline__ int paged_len_ok(const PagedView &v, int len) {
    const int64_t cap = (int64_t)v.max_pages << v.page_shift;
    if (len < 0 || len > cap) {
        record_error(kErrPaged);
        return 0;
    }
    return len;
}

// Keys of sequence b.
__device__ __forceinline__ int paged_len(const PagedView &v, int b) { return paged_len_ok(v, v.kv_len[b]); }

// Whether s .. e - 1 are rows of a sequence.
__device__ __forceinline__ bool paged_starts_ok(const PagedView &v, int s, int e) {
    if (s >= 0 && e >= s && e <= v.n_tokens) return true;
    record_error(kErrPaged);
    return false;
}

// First token row, token count and keys of sequence b (its loads go out together).
__device__ __forceinline__ void paged_seq(const PagedView &v, int b, int &start, int &count, int &len) {
    int s = b, e = b + 1;
    if (v.q_start) {
        s = v.q_start[b];
        e = v.q_start[b + 1];
    }
    len = paged_len(v, b);
    start = s;
    count = e - s;
    if (!paged_starts_ok(v, s, e)) start = count = 0;
}

// The pool row (128 values) of page entry `entry` of sequence b for global kv
// head j, slot 0; -1 when the table names a page that is not there.
__device__ __forceinline__ int64_t paged_row(const PagedView &v, int b, int entry, int j) {
    const int page = v.table[b * v.table_stride + entry];
    if (page < 0 || page >= v.n_pages) {
        record_error(kErrPaged);
        return -1;
    }
    const int sh = j / v.nkv_s, jl = j % v.nkv_s;
    return (((int64_t)sh * v.n_pages + page) * v.nkv_s + jl) << v.page_shift;
}

// 2^x by the special-function unit (relative error 2^-22; 2^-inf = 0).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- append ----------------------------------------------------------------
//
// q' = R(p) q, and for the token's slot of the cache K = bf16(R(p) k), V =
// bf16(v), where R(p) turns the pair (x[e], x[e + 64]) by p * rope_base^(-2e/128)
// (RoFormer's rotation, half-split pairing; TPL_ROPE) or is the identity.
// A pass over memory: every value is read once and written once, so HBM is
// the bound and the rotation has to stay hidden behind the loads.  One CTA
// takes one token, several when a token has few heads, or a part of its heads
// when there are few tokens: the 64 angles of a token are formed once, in turns
// and in fp64 (far positions are thousands of turns, of which only the fraction
// counts), shared by all heads, and evaluated while the CTA's first loads are
// in flight.  A work item is 16 bytes of a row's first half with the 16 bytes
// of the second half they are turned with.
// 4 warps with up to 6 items a thread measured best (bf16, 64/8 heads, 16k
// tokens: 105 us against 119 us with 8 warps and 111 us with up to 8 items;
// 32/32 heads: 96, 103 and 101 us).

constexpr int kAppendThreads = 128;
constexpr int kAppendItems = 6;   // items in flight per thread
constexpr int kAppendTokens = 8;  // tokens per CTA at most

struct AppendArgs {
    PagedView v;
    const void *q, *k, *kv;  // tokens x heads x 128 (kv: the values)
    void *q_out;             // NULL: no q
    int64_t q_ts, q_hs, qo_ts, qo_hs, k_ts, k_hs, v_ts, v_hs;  // strides in elements
    __nv_bfloat16 *kc, *vc;
    int nq;                  // query heads (0: no q)
    int rope;
    int tokens_per_cta;      // 1 when a token's items are spread over several CTAs
    int items_per_cta;       // of a token
    double turns[64];        // rope_base^(-2e/128) / (2 pi)
};

template <typename T>
struct AppendIo;
template <>
struct AppendIo<float> {
    static constexpr int N = 4;  // values per 16 bytes
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[4]) {
        x[0] = __uint_as_float(u.x);
        x[1] = __uint_as_float(u.y);
        x[2] = __uint_as_float(u.z);
        x[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
        return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    }
    static __device__ __forceinline__ void store_bf16(__nv_bfloat16 *p, const float (&x)[4]) {
        *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
    }
};
template <>
struct AppendIo<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, float (&x)[8]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = bf16lo(w[i]);
            x[2 * i + 1] = bf16hi(w[i]);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                          pack_bf16x2(x[6], x[7]));
    }
    static __device__ __forceinline__ void store_bf16(__nv_bfloat16 *p, const float (&x)[8]) {
        *reinterpret_cast<uint4 *>(p) = pack(x);
    }
};

// MANY: several tokens per CTA.
template <typename T, bool MANY>
__global__ void __launch_bounds__(kAppendThreads) paged_append_kernel(const __grid_constant__ AppendArgs a) {
    using Io = AppendIo<T>;
    constexpr int N = Io::N;
    constexpr int IPH = 64 / N;  // items per head
    constexpr int TOKENS = MANY ? kAppendTokens : 1;
    __shared__ float s_cos[TOKENS][64], s_sin[TOKENS][64];
    __shared__ int s_seq[TOKENS], s_pos[TOKENS];
    __shared__ int64_t s_row[TOKENS];  // the token's slot in the pages of head 0; -1: none
    const int tok0 = MANY ? blockIdx.x * a.tokens_per_cta : blockIdx.x;
    const int ntok = MANY ? min(a.tokens_per_cta, a.v.n_tokens - tok0) : 1;
    const int nkv = a.v.nkv;
    const int per_tok = (a.nq + 2 * nkv) * IPH;
    const int i0 = blockIdx.y * a.items_per_cta, i1 = MANY ? ntok * per_tok : min(per_tok, i0 + a.items_per_cta);
    if (threadIdx.x < TOKENS) s_seq[threadIdx.x] = -1;
    __syncthreads();
    pdl_wait();
    pdl_trigger();

    // item -> token of the CTA, head (query, key, value), first of its values
    auto split = [&](int item, int &tk, int &h, int &e) {
        tk = MANY ? item / per_tok : 0;
        if (MANY) item -= tk * per_tok;
        h = item / IPH;
        e = item % IPH * N;
    };
    auto source = [&](int item) -> const uint4 * {
        int tk, h, e;
        split(item, tk, h, e);
        const int64_t tok = tok0 + tk;
        const T *p;
        if (h < a.nq) p = static_cast<const T *>(a.q) + tok * a.q_ts + h * a.q_hs;
        else if (h < a.nq + nkv) p = static_cast<const T *>(a.k) + tok * a.k_ts + (h - a.nq) * a.k_hs;
        else p = static_cast<const T *>(a.kv) + tok * a.v_ts + (h - a.nq - nkv) * a.v_hs;
        return reinterpret_cast<const uint4 *>(p + e);
    };
    uint4 lo[kAppendItems], hi[kAppendItems];
#pragma unroll
    for (int r = 0; r < kAppendItems; ++r) {
        const int item = i0 + threadIdx.x + r * kAppendThreads;
        if (item < i1) {
            const uint4 *p = source(item);
            lo[r] = p[0];
            hi[r] = p[4 * sizeof(T)];  // 64 values on
        }
    }

    // the tokens' sequences: every thread looks at some of them
    if (a.v.q_start) {
        for (int b = threadIdx.x; b < a.v.n_seqs; b += kAppendThreads) {
            const int s = a.v.q_start[b], e = a.v.q_start[b + 1];
            if (!paged_starts_ok(a.v, s, e)) continue;  // (reported though none of its rows may be this CTA's)
            for (int x = max(s, tok0); x < min(e, tok0 + ntok); ++x) atomicMax(&s_seq[x - tok0], b);
        }
    } else if (threadIdx.x < ntok) {
        s_seq[threadIdx.x] = tok0 + threadIdx.x;
    }
    __syncthreads();
    // position and slot of token x; -1: a row of no sequence or an inactive one, and no page
    auto place = [&](int x, int &pos, int64_t &row) {
        const int b = s_seq[x];
        pos = -1;
        row = -1;
        if (b < 0) return;
        int start, count, len;
        paged_seq(a.v, b, start, count, len);
        if (count > 0) pos = len - count + (tok0 + x - start);
        if (pos < 0) return;
        row = paged_row(a.v, b, pos >> a.v.page_shift, 0);  // head 0 of shard 0
        if (row >= 0) row += pos & ((1 << a.v.page_shift) - 1);
    };
    int pos0 = 0;
    int64_t row0 = 0;
    if (MANY) {
        if (threadIdx.x < ntok) place(threadIdx.x, s_pos[threadIdx.x], s_row[threadIdx.x]);
        __syncthreads();
    } else {
        place(0, pos0, row0);
        if (pos0 < 0) return;
    }
    if (a.rope) {
        for (int x = threadIdx.x; x < ntok * 64; x += kAppendThreads) {
            const double turn = (double)(MANY ? s_pos[x / 64] : pos0) * a.turns[x % 64];
            float s, c;
            sincospif((float)(2.0 * (turn - rint(turn))), &s, &c);
            s_cos[x / 64][x % 64] = c;
            s_sin[x / 64][x % 64] = s;
        }
        __syncthreads();
    }

    for (int base = i0 + threadIdx.x; base < i1; base += kAppendItems * kAppendThreads) {
        if (base != i0 + (int)threadIdx.x) {
#pragma unroll
            for (int r = 0; r < kAppendItems; ++r) {
                const int item = base + r * kAppendThreads;
                if (item < i1) {
                    const uint4 *p = source(item);
                    lo[r] = p[0];
                    hi[r] = p[4 * sizeof(T)];
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kAppendItems; ++r) {
            const int item = base + r * kAppendThreads;
            if (item >= i1) break;
            int tk, h, e;
            split(item, tk, h, e);
            if (MANY && s_pos[tk] < 0) continue;
            const int64_t slot = MANY ? s_row[tk] : row0;
            float x[N], y[N];
            Io::unpack(lo[r], x);
            Io::unpack(hi[r], y);
            if (a.rope && h < a.nq + nkv) {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float c = s_cos[tk][e + i], s = s_sin[tk][e + i], x0 = x[i];
                    x[i] = x0 * c - y[i] * s;
                    y[i] = y[i] * c + x0 * s;
                }
            }
            if (h < a.nq) {
                T *p = static_cast<T *>(a.q_out) + (int64_t)(tok0 + tk) * a.qo_ts + h * a.qo_hs + e;
                *reinterpret_cast<uint4 *>(p) = Io::pack(x);
                *reinterpret_cast<uint4 *>(p + 64) = Io::pack(y);
            } else if (slot >= 0) {
                const bool is_k = h < a.nq + nkv;
                const int j = h - a.nq - (is_k ? 0 : nkv);
                const int sh = j / a.v.nkv_s, jl = j % a.v.nkv_s;
                const int64_t row = slot + ((((int64_t)sh * a.v.n_pages * a.v.nkv_s) + jl) << a.v.page_shift);
                __nv_bfloat16 *p = (is_k ? a.kc : a.vc) + row * 128 + e;
                Io::store_bf16(p, x);
                Io::store_bf16(p + 64, y);
            }
        }
    }
}

}  // namespace tpl
