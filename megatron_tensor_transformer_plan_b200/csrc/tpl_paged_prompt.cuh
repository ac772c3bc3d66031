// Attention of many query rows over a paged cache, on the 5th-generation
// tensor cores: the prompts of a ragged batch (causal, with a window and
// sinks), and the common prefix of a decode batch.
//
// A row is one (token, query head); the g heads that share a kv head are rows
// of the same tile (row = token * g + head), so every key is read once for
// all of them.  An item is 256 rows of one kv head (two tiles of 128: tensor
// memory holds S and O of both) against the tiles of 128 keys that any of its
// rows sees.  The items' key tiles are laid end to end, kv head by kv head, and
// CTA c of G takes an equal contiguous range of them, so the SMs finish
// together whatever the lengths are and a few rows against a long cache still
// fill the GPU.  An item that is cut leaves one partial (max, sum,
// unnormalised output) per CTA in the workspace; a second kernel joins them.
// Neighbouring CTAs work on the same kv head, so its keys come from L2.
//
// 12 warps:
//   0     TMA producer: K and V tiles in turn into a ring, a lane per page
//         part (64 dims of at most 128 keys of one page), no multicast;
//   1, 3  MMA issuers of tile 0 and of tile 1 (warp 1 owns the tensor memory);
//   2     replaces the values of keys that no row sees by zero (0 * NaN is NaN)
//         in the tiles that have such keys, before the MMA reads them;
//   4-7   softmax of tile 0, 8-11 softmax of tile 1: one thread per row.
// A key tile is taken in two halves of 64 keys: S of one half is formed while
// the softmax works on the other, and the two tiles alternate, so that neither
// the tensor cores nor the special-function units wait for a round trip.
// S = Q K^T reads Q (bf16, or bf16 hi + lo when q is fp32: two products) and K
// from shared memory; P replaces half of S in tensor memory as bf16; O += P V.
// P has one bf16 part: with o rounded to bf16 anyway, the two roundings are of
// the same size (up to 2^-8 of each term against up to 2^-8 of the sum); the
// denominator adds the unrounded fp32 terms.  Against 64 bits o is off by 2.2e-3
// of its norm, of which its own rounding is 1.7e-3.
// The bound is the larger of the two products on the tensor cores and one
// exponential per (row, key): 128 x 128 of them take the SM's 16 lanes of the
// special-function unit as long as the two products take.
// Measured: 4096 tokens after 4096 keys, 64/8 heads, bf16: 826 us (1000 TFLOP/s,
// the clock held down by the power limit; 730 us before that sets in); with fp32
// queries, 1.5 times the products, 950 us before that.  S with
// N = 64 costs 48 cycles a product instead of 32 (its A operand is read from
// shared memory each time), which the half tile in flight more than returns
// (S of 128 keys and none in flight: 904 us).
//
// Every wait is bounded (2 s); on a timeout the roles stop, the error word is
// set, copies in flight are waited for (bounded) and TMEM is released.
#pragma once

#include <cuda.h>

#include "tpl_attn_tc.cuh"
#include "tpl_paged.cuh"

namespace tpl {

constexpr int kPtKeys = 128;                   // keys per tile
constexpr int kPtHalf = kPtKeys * 128;         // 128 rows x 64 dims, bf16: 16 KB
constexpr int kPtTile = 2 * kPtHalf;           // one K, V or Q tile: 32 KB
constexpr int kPtThreads = 384;
// Key tiles per CTA at least.  Prompts: any.  With 1, 2 and 4: 3 of up to 37 tokens after up
// to 900 keys 20.8, 24.4 and 26.6 us, 3 of 37 after 900 each 27.4, 23.1 and 24.5, one of 100
// after 100 20.4, 19.1 and 27.5, 4 of 64 after 1 17.9, 24.2 and 37.9, 512 after none 29.0,
// 28.5 and 33.9, 16 after 9000 the same.  A prefix: every cut of an item is one more partial
// of all its rows to write and join.  With 1, 2, 4, 6 and 8 (a call, two keys of its own per
// sequence): 5 sequences, 1536 keys, 32/32 heads 26.7, 26.8, 19.9, 21.3 and 27.8 us; 16, 4096,
// 64/8 32.5, 32.2, 22.9, 24.0 and 25.6; 32, 2048, 40/8 32.0, 20.8, 22.2, 29.0 and 29.1; 8,
// 1024, 16/2 17.1, 15.9, 16.8, 21.4 and 21.4; 3, 16384, 32/8 38.0, 37.9, 37.9, 38.0 and 30.2;
// 64, 8192, 64/8 the same.
constexpr int kPtMinTiles = 1, kPtMinTilesPrefix = 4;
constexpr uint32_t kPtO = 0, kPtS = 256;       // TMEM columns: O of tile t at 128 t, S at 256 + 128 t

template <bool QF32>
struct PtSmem {
    static constexpr int QPARTS = QF32 ? 2 : 1;
    static constexpr int NST = QF32 ? 3 : 5;   // ring stages of one tile; odd: see v_ready
    static constexpr int Q = 2 * QPARTS * kPtTile;
    static constexpr int BAR = 1024;
    static constexpr size_t BYTES = (size_t)Q + NST * kPtTile + BAR;
    static_assert(BYTES <= 232448, "shared memory per block");
    static_assert(NST % 2 == 1, "K and V alternate on every stage");
};

struct PagedPromptArgs {
    CUtensorMap tm_k, tm_v;  // pool rows x 128, boxes of 64 dims x min(128, page) rows
    PagedView v;
    const void *q;           // [n_tokens] rows
    int64_t q_ts, q_hs;
    int nq, g, tb;           // tb = tokens per tile = 128 / g
    int window, sinks;
    int shared;              // > 0: the common prefix of this many keys (rows = sequences)
    float scale_log2;
    __nv_bfloat16 *o;        // [n_tokens][nq * 128]
    float *lse;              // [n_tokens][nq] or NULL
    // partials: slots of rows x 128 floats and rows x 2; prompts: slot 2 c + (not the
    // CTA's first segment); prefix: slot item + c
    float *part_o, *part_ml;
    int part_rows;           // rows per slot
    int G;                   // CTAs that take part (0: decided at the device)
    unsigned *ready;         // prefix: set once all that came before this kernel is there (pdl_pass_on)
    int4 *cut;               // [grid] prompts: {first token, row tokens, kv head, parts} of the item CTA c is the first of
};

// One item: 2 * tb tokens of a sequence against the key tiles they see.
struct PtItem {
    int row0, ntok;      // first row of q, tokens
    int p0;              // position of the first token
    int len, lo, sk;     // some row sees key j: j < len && (j >= lo || j < sk)
    int nst, ft, ntk;    // key tiles: 0 .. nst-1, then ft ..; ntk of them
    __device__ __forceinline__ int tile(int i) const { return i < nst ? i : ft + i - nst; }
};

__device__ __forceinline__ int pt_items(const PagedPromptArgs &a, int count) { return (count + 2 * a.tb - 1) / (2 * a.tb); }

// The first key of position p's window (p may lie below 0).
__device__ __forceinline__ int pt_window(const PagedPromptArgs &a, int p) {
    return a.window > 0 && p >= a.window ? p - a.window + 1 : 0;
}

__device__ __forceinline__ PtItem pt_item(const PagedPromptArgs &a, int len, int start, int count, int it) {
    PtItem x;
    const int t0 = it * 2 * a.tb;
    x.row0 = start + t0;
    x.ntok = min(2 * a.tb, count - t0);
    if (a.shared > 0) {
        x.p0 = a.shared;
        x.len = min(a.shared, len);
        x.lo = x.sk = x.nst = x.ft = 0;
        x.ntk = (a.shared + kPtKeys - 1) / kPtKeys;
        return x;
    }
    x.p0 = len - count + t0;
    x.len = max(0, x.p0 + x.ntok);
    x.lo = pt_window(a, x.p0);
    x.sk = min(a.sinks, x.lo);
    x.nst = (x.sk + kPtKeys - 1) / kPtKeys;
    x.ft = max(x.lo / kPtKeys, x.nst);
    // rows that see no key still take one (masked) tile, which gives them zeros
    x.ntk = max(1, x.nst + max(0, (int)(((int64_t)x.len + kPtKeys - 1) / kPtKeys) - x.ft));
    return x;
}

// Keys of the longest sequence behind a prefix, by the whole warp; `len`: lane's sequence's.
// A prefix that no sequence fills is read, and its values are taken, up to there: what lies
// behind it may be anything, and 0 * NaN is NaN.  The two warps that need it (the loads and
// the check of the values) ask; the softmax masks by each row's own length.  One sequence
// that goes on behind the prefix is enough to know, and is most often among the first 32.
__device__ __forceinline__ int pt_longest(const PagedPromptArgs &a, int lane, int len) {
    int top = paged_len_ok(a.v, len);
    if (__any_sync(0xffffffffu, top >= a.shared)) return a.shared;
#pragma unroll 1
    for (int b = lane + 32; b < a.v.n_seqs; b += 32) top = max(top, paged_len(a.v, b));
    return __reduce_max_sync(0xffffffffu, top);
}

// Walks a CTA's segments in order; every role walks on its own.
struct PtWalk {
    int64_t u, u1;
    int j, b, it;        // kv head, sequence, item of the sequence
    int start, count, len;  // its tokens and keys (a prefix: see pt_longest)
    int done;            // key tiles of the item before u
    int idx;             // items before this one, over all kv heads (prefix mode)
    PtItem x;
    int i0, n;           // this segment: key tiles i0 .. i0 + n - 1 of the item
    bool first;          // the CTA's first segment

    __device__ __forceinline__ void open(const PagedPromptArgs &a) {
        x = pt_item(a, len, start, count, it);
        i0 = done;
        n = (int)min((int64_t)(x.ntk - done), u1 - u);
    }
    __device__ __forceinline__ void tokens(const PagedPromptArgs &a) {
        if (a.shared > 0) {
            start = 0;
            count = a.v.n_tokens;
        } else {
            paged_seq(a.v, b, start, count, len);
        }
    }
    __device__ __forceinline__ bool next(const PagedPromptArgs &a) {
        u += n;
        if (u >= u1) return false;
        first = false;
        done = 0;
        ++idx;
        if (++it == pt_items(a, count)) {
            it = 0;
            const int ns = a.shared > 0 ? 1 : a.v.n_seqs;
            do {
                if (++b == ns) {
                    b = 0;
                    ++j;
                }
                tokens(a);
            } while (count == 0);
        }
        open(a);
        return true;
    }
    __device__ __forceinline__ bool whole() const { return i0 == 0 && n == x.ntk; }
};

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Two fp32 values at a time: the fma and add units take packed pairs.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// True in one lane of the warp, always the same one.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{ .reg .pred P; elect.sync _|P, 0xffffffff; selp.u32 %0, 1, 0, P; }" : "=r"(p));
    return p != 0;
}

// The n lowest bits (none for n <= 0, all from n = 32 on).
__device__ __forceinline__ uint32_t low_bits(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Uses of a loaded row stay behind the wait for it.
__device__ __forceinline__ void tmem_ld_done(float *v) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]),
                          "+f"(v[i + 6]), "+f"(v[i + 7]));
}

template <bool QF32>
__global__ void __launch_bounds__(kPtThreads, 1) paged_prompt_kernel(const __grid_constant__ PagedPromptArgs a) {
    using SM = PtSmem<QF32>;
    constexpr int NST = SM::NST;
    extern __shared__ __align__(1024) unsigned char pt_raw[];
    unsigned char *sm = pt_raw;
    if (smem_u32(sm) & 1023u) {  // (the whole grid: the swizzled tiles need 1 KB alignment)
        if (threadIdx.x == 0) record_error(8u);
        pdl_wait();
        return;
    }
    unsigned char *s_q = sm;              // [tile][part][half][128 rows][128 B]
    unsigned char *ring = sm + SM::Q;
    // A stage holds a K and a V tile in turn (NST is odd).  Each kind has its own barriers
    // for having landed, with a phase per two laps: a wait names a phase by its parity, so
    // whoever waits for one kind must not depend on having seen the other.
    uint64_t *full_k = reinterpret_cast<uint64_t *>(ring + NST * kPtTile);  // [NST]
    uint64_t *full_v = full_k + NST;      // [NST]
    uint64_t *empty = full_v + NST;       // [NST] tile read by its last MMA
    uint64_t *v_ready = empty + NST;      // [NST] V tile checked
    uint64_t *q_ready = v_ready + NST;    // [2]
    uint64_t *s_full = q_ready + 2;       // [2 tiles][2 halves]
    uint64_t *p_full = s_full + 4;        // [2][2]
    uint64_t *pv_done = p_full + 4;       // [2]
    uint64_t *o_full = pv_done + 2;       // [2]
    uint64_t *o_empty = o_full + 2;       // [2]
    uint64_t *fin = o_empty + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(fin + 1);
    volatile int *s_fail = reinterpret_cast<volatile int *>(tmem_slot + 1);
    int *s_issued = const_cast<int *>(s_fail) + 1;
    int *s_where = s_issued + 1;          // [7] start of this CTA's range: j, b, item, tiles before; b's tokens and keys
    long long *s_sum = reinterpret_cast<long long *>((reinterpret_cast<uintptr_t>(s_where + 7) + 7) & ~(uintptr_t)7);
    static_assert((4 * NST + 17) * 8 + 56 + 16 + kPtThreads / 32 * 8 <= SM::BAR, "barrier area");

    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NST; ++s) {
            mbar_init(&full_k[s], 1);
            mbar_init(&full_v[s], 1);
            mbar_init(&empty[s], 2);
            mbar_init(&v_ready[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&q_ready[t], 4);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&s_full[2 * t + h], 1);
                mbar_init(&p_full[2 * t + h], 4);
            }
            mbar_init(&pv_done[t], 1);
            mbar_init(&o_full[t], 1);
            mbar_init(&o_empty[t], 4);
        }
        mbar_init(fin, 2);
        *s_fail = 0;
        *s_issued = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    if (a.ready && cta == 0 && threadIdx.x == 0) pdl_pass_on(a.ready);
    pdl_trigger();

    // ---- this CTA's range of the key tiles ----
    int64_t U1;  // key tiles of one kv head
    int lane_len = 0;  // a prefix: keys of sequence `lane`
    if (a.shared > 0) {
        if ((warp == 0 || warp == 2) && lane < a.v.n_seqs) lane_len = a.v.kv_len[lane];
        U1 = (int64_t)pt_items(a, a.v.n_tokens) * ((a.shared + kPtKeys - 1) / kPtKeys);
    } else {
        // the sequences' items, tokens and keys; then each thread sums a run of items
        const int ns = a.v.n_seqs;
        int *s_item = reinterpret_cast<int *>(ring);  // [n_seqs + 1] items before sequence b
        int *s_start = s_item + kPagedMaxSeqs + 1, *s_count = s_start + kPagedMaxSeqs, *s_len = s_count + kPagedMaxSeqs;
        constexpr int PT = (kPagedMaxSeqs + kPtThreads - 1) / kPtThreads;
        const int per = (ns + kPtThreads - 1) / kPtThreads;
        int mine[PT], cnt = 0;
#pragma unroll
        for (int x = 0; x < PT; ++x) {
            const int b = threadIdx.x * per + x;
            mine[x] = 0;
            if (x < per && b < ns) {
                int start, count, len;
                paged_seq(a.v, b, start, count, len);
                s_start[b] = start;
                s_count[b] = count;
                s_len[b] = len;
                mine[x] = pt_items(a, count);
            }
            cnt += mine[x];
        }
        auto scan = [&](long long val) -> long long {  // exclusive prefix over the CTA's threads
            long long inc = val;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long t = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += t;
            }
            if (lane == 31) s_sum[warp] = inc;
            __syncthreads();
            long long at = inc - val;
#pragma unroll
            for (int w = 0; w < kPtThreads / 32; ++w) at += w < warp ? s_sum[w] : 0;
            return at;
        };
        int at = (int)scan(cnt);
#pragma unroll
        for (int x = 0; x < PT; ++x) {
            const int b = threadIdx.x * per + x;
            if (x < per && b < ns) {
                s_item[b] = at;
                at += mine[x];
                if (b == ns - 1) s_item[ns] = at;
            }
        }
        __syncthreads();
        const int items = s_item[ns];
        const int run = (items + kPtThreads - 1) / kPtThreads;
        const int k0 = min(items, (int)threadIdx.x * run), k1 = min(items, k0 + run);
        // items k0 .. k1 - 1: their sequence, then their key tiles
        auto walk = [&](auto &&visit) {
            if (k0 >= k1) return;
            int l = 0, r = ns - 1;  // the last sequence that begins at or before item k0
            while (l < r) {
                const int mid = (l + r + 1) >> 1;
                if (s_item[mid] <= k0) l = mid;
                else r = mid - 1;
            }
            int b = l;
            for (int k = k0; k < k1; ++k) {
                while (k >= s_item[b + 1]) ++b;
                visit(b, k - s_item[b], pt_item(a, s_len[b], s_start[b], s_count[b], k - s_item[b]).ntk);
            }
        };
        long long tiles = 0;
        walk([&](int, int, int ntk) { tiles += ntk; });
        long long before = scan(tiles);
        __syncthreads();
        if (threadIdx.x == kPtThreads - 1) s_sum[0] = before + tiles;
        __syncthreads();
        U1 = s_sum[0];
        const int64_t U = U1 * a.v.nkv;
        const int G = (int)min((int64_t)gridDim.x, max((int64_t)1, (U + kPtMinTiles - 1) / kPtMinTiles));
        if (cta < G && U > 0) {
            const int64_t u0 = paged_cut(U, G, cta);
            const int j = (int)paged_div(u0, U1);
            const int64_t rel = u0 - j * U1;
            if (rel >= before && rel < before + tiles) {
                long long t = before;
                walk([&](int b, int it, int ntk) {
                    if (rel >= t && rel < t + ntk) {
                        s_where[0] = j;
                        s_where[1] = b;
                        s_where[2] = it;
                        s_where[3] = (int)(rel - t);
                        s_where[4] = s_start[b];
                        s_where[5] = s_count[b];
                        s_where[6] = s_len[b];
                    }
                    t += ntk;
                });
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ring is TMA's from here on
        __syncthreads();
    }
    const int64_t U = U1 * a.v.nkv;
    const int G = a.G > 0 ? a.G : (int)min((int64_t)gridDim.x, max((int64_t)1, (U + kPtMinTiles - 1) / kPtMinTiles));
    const bool busy = cta < G && U > 0;
    if (threadIdx.x == 128 && a.cut) a.cut[cta] = make_int4(0, 0, 0, 0);  // the thread that may fill it in below

    PtWalk w;
    if (busy) {
        w.u = paged_cut(U, G, cta);
        w.u1 = paged_cut(U, G, cta + 1);
        w.first = true;
        if (a.shared > 0) {
            const int items = pt_items(a, a.v.n_tokens), NT = (a.shared + kPtKeys - 1) / kPtKeys;
            w.idx = (int)paged_div(w.u, NT);
            w.done = (int)(w.u - (int64_t)w.idx * NT);
            w.j = w.idx / items;
            w.it = w.idx - w.j * items;
            w.b = 0;
            w.len = warp == 0 || warp == 2 ? pt_longest(a, lane, lane_len) : a.shared;
            w.tokens(a);
        } else {
            w.j = s_where[0];
            w.b = s_where[1];
            w.it = s_where[2];
            w.done = s_where[3];
            w.start = s_where[4];
            w.count = s_where[5];
            w.len = s_where[6];
            w.idx = 0;  // (a prefix's only)
        }
        w.open(a);
    }

    if (busy && warp == 0) {
        // ---- TMA producer: K and V tiles in turn.  The pages of 32 parts (whole tiles)
        //      are looked up at once, a batch ahead. ----
        const int box_shift = min(a.v.page_shift, 7);
        const int nsub = kPtKeys >> box_shift;  // parts of a tile: at most 8
        const int half = lane / nsub, sub = lane % nsub;  // this lane's copy (half < 2)
        const int batch = 32 / nsub;            // tiles per lookup
        int e = 0;
        bool ok = true;
        do {
            const PtItem &x = w.x;
            const int seq = a.shared > 0 ? 0 : w.b, i1 = w.i0 + w.n;
            const int64_t jrow = (int64_t)(w.j / a.v.nkv_s) * a.v.n_pages * a.v.nkv_s + w.j % a.v.nkv_s;
            // the page of part lane % nsub of tile i0 + lane / nsub: -1 when no key of it is seen
            auto lookup = [&](int i0) {
                const int i = i0 + lane / nsub, key = x.tile(min(i, i1 - 1)) * kPtKeys + ((lane % nsub) << box_shift);
                const bool want = i < i1 && key < x.len && (key + (1 << box_shift) > x.lo || key < x.sk);
                int page = -1;
                if (want) page = max(a.v.table[seq * a.v.table_stride + (key >> a.v.page_shift)], -2);
                return want && page < 0 ? -2 : page;
            };
            int ahead = lookup(w.i0);
            for (int ib = w.i0; ok && ib < i1; ib += batch) {
                int page = ahead;
                if (ib + batch < i1) ahead = lookup(ib + batch);
                if (page == -2 || page >= a.v.n_pages) {
                    record_error(kErrPaged);
                    page = 0;
                }
                const int base = page < 0 ? -1 : (int)((jrow + (int64_t)page * a.v.nkv_s) << a.v.page_shift);
                for (int i = ib; ok && i < min(ib + batch, i1); ++i) {
                    int row = __shfl_sync(0xffffffffu, base, (i - ib) * nsub + sub);
                    const bool want = half < 2 && row >= 0;
                    row += (x.tile(i) * kPtKeys + (sub << box_shift)) & ((1 << a.v.page_shift) - 1);
                    const unsigned bytes = (unsigned)__popc(__ballot_sync(0xffffffffu, want)) << (box_shift + 7);
                    for (int kv = 0; ok && kv < 2; ++kv) {
                        const int s = e % NST;
                        uint64_t *full = kv ? &full_v[s] : &full_k[s];
                        bool go = true;
                        if (lane == 0) {
                            go = mbar_wait(&empty[s], ((unsigned)(e / NST) & 1u) ^ 1u);
                            if (go) mbar_expect_tx(full, bytes);
                        }
                        ok = __all_sync(0xffffffffu, go);
                        if (!ok) break;
                        if (want)
                            tma_load_2d(ring + s * kPtTile + half * kPtHalf + (sub << (box_shift + 7)),
                                        kv ? &a.tm_v : &a.tm_k, 64 * half, row, full);
                        ++e;
                    }
                }
            }
        } while (ok && w.next(a));
        if (!ok) *s_fail = 1;
        if (lane == 0) *s_issued = e;
    } else if (busy && (warp == 1 || warp == 3)) {
        // ---- MMA issuers: warp 1 the products of tile 0, warp 3 those of tile 1.  The whole
        //      warp walks and one elected lane issues, so that the products' operands stay
        //      in uniform registers. ----
        const int t = warp >> 1;
        constexpr uint32_t IDESC_S = umma_idesc(128, kPtKeys / 2);
        constexpr uint32_t IDESC_PV = umma_idesc(128, 128) | (1u << 16);  // B (V) MN-major
        constexpr unsigned TILE16 = kPtTile >> 4, HALF16 = kPtHalf >> 4, ROWS16 = 64 * 128 >> 4;  // (descriptors count 16 bytes)
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dq = umma_desc(smem_u32(s_q)) + t * SM::QPARTS * TILE16, dk0 = umma_desc(smem_u32(ring)),
                       dv0 = umma_desc_lbo(smem_u32(ring), kPtHalf);
        const uint32_t d_o = tm + kPtO + 128u * t, d_s = tm + kPtS + 128u * t;
        int sk = 0, sv = 1;                // ring stages of the next K and V
        unsigned lk = 0, lv = 0;           // and their laps
        unsigned n_p = 0, n_q = 0;         // phases of p_full, and of q_ready / o_empty
        bool ok = true;
        auto wait = [&](uint64_t *bar, unsigned parity) { ok = ok && __all_sync(0xffffffffu, mbar_wait(bar, parity & 1u)); };
        auto commit = [&](uint64_t *bar) {
            if (elect_one()) umma_commit(bar);
        };
        auto issue_s = [&](int h) {  // 64 keys of S = Q K^T
            const uint64_t dk = dk0 + sk * TILE16 + h * ROWS16;
            if (elect_one()) {
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
                for (int kk = 0; kk < 8; ++kk) {
                    const unsigned off = (kk >> 2) * HALF16 + 2 * (kk & 3);
                    umma(d_s + 64u * h, dq + off, dk + off, IDESC_S, kk > 0 ? 1u : 0u);
                    if (QF32) umma(d_s + 64u * h, dq + TILE16 + off, dk + off, IDESC_S, 1u);
                }
                umma_commit(&s_full[2 * t + h]);
                if (h == 1) umma_commit(&empty[sk]);
            }
        };
        auto issue_pv = [&](int h, bool acc, bool last) {  // O += P V over 64 keys
            const uint64_t dv = dv0 + sv * TILE16 + h * ROWS16;
            if (elect_one()) {
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll
                for (int ks = 0; ks < kPtKeys / 32; ++ks)
                    umma_ts(d_o, d_s + 64u * h + 8 * ks, dv + ks * (2048 >> 4), IDESC_PV, (acc || ks > 0) ? 1u : 0u);
                umma_commit(&pv_done[t]);
                if (h == 1) umma_commit(&empty[sv]);
                if (h == 1 && last) umma_commit(&o_full[t]);
            }
        };
        // a stage on: NST is odd, so K and V alternate on every stage
        auto step = [&](int &stage, unsigned &lap) {
            stage += 2;
            if (stage >= NST) {
                stage -= NST;
                ++lap;
            }
        };
        PtWalk nx;  // the segment after this one: looked up while this one is worked on
        do {
            nx = w;
            const int another = nx.next(a);
            const bool mine = __shfl_sync(0xffffffffu, (int)(t == 0 || w.x.ntok > a.tb), 0);
            const int n = __shfl_sync(0xffffffffu, w.n, 0);
            if (mine) wait(&q_ready[t], n_q);
            wait(&full_k[sk], lk >> 1);
            if (ok && mine) issue_s(0), issue_s(1);
            if (ok && !mine) commit(&empty[sk]);  // (an item of one tile: its stages need this warp's word too)
            step(sk, lk);
            for (int i = 0; ok && i < n; ++i) {
                const bool more = i < n - 1;
                wait(&v_ready[sv], lv >> 1);
                if (more) wait(&full_k[sk], lk >> 1);
                if (mine) {
                    if (i == 0) wait(&o_empty[t], n_q ^ 1u);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        wait(&p_full[2 * t + h], n_p);
                        if (!ok) break;
                        issue_pv(h, i > 0 || h > 0, !more);
                        if (more) issue_s(h);
                    }
                    ++n_p;
                } else if (ok) {
                    commit(&empty[sv]);
                    if (more) commit(&empty[sk]);
                }
                step(sv, lv);
                if (more) step(sk, lk);
            }
            if (mine) ++n_q;
            w = nx;
            if (!__shfl_sync(0xffffffffu, another, 0)) break;
        } while (ok);
        if (!ok) *s_fail = 1;
        commit(fin);
        if (!mbar_wait(fin, 0)) *s_fail = 1;
    } else if (busy && warp == 2) {
        // ---- values of keys that no row sees become zero; the next segment's queries are
        //      brought into L2 while this one's keys are worked on ----
        int e = 1;
        bool ok = true, another;
        do {
            const PtItem x = w.x;
            PtWalk nx = w;
            another = nx.next(a);
            if (another) {
                const int size = QF32 ? 4 : 2, lines = size;  // 128-byte lines of a row
                for (int k = lane; k < nx.x.ntok * a.g * lines; k += 32) {
                    const int rk = k / lines;
                    const int64_t o = (nx.x.row0 + rk / a.g) * a.q_ts + (nx.j * a.g + rk % a.g) * a.q_hs;
                    prefetch_l2(static_cast<const char *>(a.q) + o * size + 128 * (k % lines));
                }
            }
            for (int i = w.i0; ok && i < w.i0 + w.n; ++i, e += 2) {
                const int s = e % NST;
                ok = __all_sync(0xffffffffu, mbar_wait(&full_v[s], (unsigned)((e / NST) >> 1) & 1u));
                if (!ok) break;
                const int k0 = x.tile(i) * kPtKeys;
                if (!(k0 + kPtKeys <= x.len && (k0 >= x.lo || k0 + kPtKeys <= x.sk))) {
                    unsigned char *st = ring + s * kPtTile;
                    for (int r = lane; r < kPtKeys; r += 32) {
                        const int key = k0 + r;
                        if (key < x.len && (key >= x.lo || key < x.sk)) continue;
#pragma unroll
                        for (int c = 0; c < 16; ++c)
                            *reinterpret_cast<uint4 *>(st + (c >> 3) * kPtHalf + r * 128 + 16 * (c & 7)) =
                                make_uint4(0, 0, 0, 0);
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&v_ready[s]);
            }
            w = nx;
        } while (ok && another);
        if (!ok) *s_fail = 1;
    } else if (busy && warp >= 4) {
        // ---- softmax: thread = row of tile t ----
        const int t = (warp - 4) >> 2, qd = warp & 3;
        const int r = 32 * qd + lane;
        const uint32_t lane_off = (uint32_t)(32 * qd) << 16;
        const uint32_t scol = tmem + lane_off + kPtS + 128u * t, ocol = tmem + lane_off + kPtO + 128u * t;
        unsigned n_s = 0, seg = 0;  // half tiles (phases of s_full and pv_done) and segments so far
        // The warp's 32 rows of a segment's q into shared memory, 128-byte swizzle: a row
        // (fp32) or two (bf16) per load, the lanes side by side, sixteen loads at a time.
        auto load_q = [&](const PtWalk &y) {
            if (t == 1 && y.x.ntok <= a.tb) return;
            unsigned char *dst = s_q + t * SM::QPARTS * kPtTile;
            const int tok = t * a.tb + r / a.g;
            const bool live = r < a.tb * a.g && tok < y.x.ntok;
            const long long off = live ? (y.x.row0 + tok) * a.q_ts + (y.j * a.g + r % a.g) * a.q_hs : -1;
            if (QF32) {
                const int half = lane >> 4, c = (lane & 15) >> 1;
#pragma unroll 1
                for (int k0 = 0; k0 < 32; k0 += 16) {
                    float4 f[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {  // (rows of no token: any address, then zeros)
                        const long long o = __shfl_sync(0xffffffffu, off, k0 + k);
                        f[k] = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + max(o, 0ll))[lane];
                        if (o < 0) f[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const int rk = 32 * qd + k0 + k;
                        unsigned char *d = dst + half * kPtHalf + rk * 128 + ((c ^ (k & 7)) << 4) + 8 * (lane & 1);
                        const uint32_t h0 = pack_bf16x2(f[k].x, f[k].y), h1 = pack_bf16x2(f[k].z, f[k].w);
                        *reinterpret_cast<uint2 *>(d) = make_uint2(h0, h1);
                        *reinterpret_cast<uint2 *>(d + kPtTile) =
                            make_uint2(pack_bf16x2(f[k].x - bf16lo(h0), f[k].y - bf16hi(h0)),
                                       pack_bf16x2(f[k].z - bf16lo(h1), f[k].w - bf16hi(h1)));
                    }
                }
            } else {
                const int half = (lane & 15) >> 3, c = lane & 7;
#pragma unroll 1
                for (int k0 = 0; k0 < 32; k0 += 32) {
                    uint4 u[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const long long o = __shfl_sync(0xffffffffu, off, k0 + 2 * k + (lane >> 4));
                        u[k] = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) + max(o, 0ll))[lane & 15];
                        if (o < 0) u[k] = make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const int rk = 32 * qd + k0 + 2 * k + (lane >> 4);
                        *reinterpret_cast<uint4 *>(dst + half * kPtHalf + rk * 128 + ((c ^ (rk & 7)) << 4)) = u[k];
                    }
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_ready[t]);
        };
        bool ok = true, another;
        PtWalk nx;  // the segment after this one: looked up while this one is worked on
        load_q(w);
        do {
            const PtItem x = w.x;
            nx = w;
            another = nx.next(a);
            if (t == 1 && x.ntok <= a.tb) {
                if (another) load_q(nx);
                w = nx;
                continue;  // (evaluates the loop's condition)
            }
            const int tok = t * a.tb + r / a.g;      // token of the item
            const int head = w.j * a.g + r % a.g;
            const bool live = r < a.tb * a.g && tok < x.ntok;
            const bool warp_live = __any_sync(0xffffffffu, live);
            const int64_t row = x.row0 + tok;
            // the last key this row sees, and the first of its window
            int p = x.p0 + tok;
            if (a.shared > 0 && live) p = min(a.shared, paged_len(a.v, (int)row)) - 1;
            const int lo = pt_window(a, p);
            // the same of all rows of this warp: tiles up to the one and from the other need no mask
            const int all_p = __reduce_min_sync(0xffffffffu, live ? p : 0x7fffffff);
            const int all_lo = __reduce_max_sync(0xffffffffu, live ? lo : 0);

            float m = -INFINITY, l = 0.f;  // running maximum (log2 units) and sum
#pragma unroll 1
            for (int i = 0; i < 2 * w.n; ++i) {
                const int h = i & 1;
                const uint32_t hcol = scol + 64u * h;
                ok = __all_sync(0xffffffffu, mbar_wait(&s_full[2 * t + h], (n_s >> 1) & 1u));
                if (!ok) break;
                ++n_s;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                if (warp_live) {
                    const int k0 = x.tile(w.i0 + (i >> 1)) * kPtKeys + 64 * h;
                    float s[64], mc[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                    tmem_ld32(hcol, s);
                    tmem_ld32(hcol + 32, s + 32);
                    tmem_ld_wait();
                    tmem_ld_done(s);
                    tmem_ld_done(s + 32);
                    if (!(k0 + 63 <= all_p && (k0 >= all_lo || k0 + 64 <= a.sinks))) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const int kc = k0 + 32 * c;  // key <= p && (key >= lo || key < sinks), a bit per key
                            const uint32_t vis = low_bits(p - kc + 1) & (~low_bits(lo - kc) | low_bits(a.sinks - kc));
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(vis >> e & 1u)) s[32 * c + e] = -INFINITY;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 64; e += 8)  // four chains: one would be latency
#pragma unroll
                        for (int c = 0; c < 4; ++c) mc[c] = max3(mc[c], s[e + c], s[e + 4 + c]);
                    const float mx = max3(fmaxf(mc[0], mc[1]), mc[2], mc[3]) * a.scale_log2;
                    // raise the running maximum only when this tile exceeds it by > 8
                    const bool need = mx > m + kAmLazy;
                    if (__any_sync(0xffffffffu, need)) {
                        const float mn = need ? mx : m;
                        const float f = need ? exp2f(m - mn) : 1.f;  // 0 on the first step (m = -inf)
                        if (i > 0) {
                            // the product of the half tile before may still be adding to O
                            // (n_s counts this one: phase n_s - 2)
                            if (!__all_sync(0xffffffffu, !*s_fail && mbar_wait(&pv_done[t], n_s & 1u))) *s_fail = 1;
                            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
                            for (int c = 0; c < 8; ++c) {
                                float v[16];
                                tmem_ld16(ocol + 16 * c, v);
                                uint32_t u[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e) u[e] = __float_as_uint(v[e] * f);
                                tmem_st16(ocol + 16 * c, u);
                            }
                        }
                        l *= f;
                        m = mn;
                    }
                    const float sub = m == -INFINITY ? 0.f : m;  // no key seen yet: every term is 2^-inf
                    const uint64_t scale2 = pack2(a.scale_log2, a.scale_log2), sub2 = pack2(-sub, -sub);
                    uint64_t l2[2] = {0, 0};
                    // P (bf16) replaces the first 32 of these 64 columns
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t u[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float x0, x1;
                            unpack2(fma2(pack2(s[32 * c + 2 * e], s[32 * c + 2 * e + 1]), scale2, sub2), x0, x1);
                            const float p0 = ex2(x0), p1 = ex2(x1);
                            l2[e & 1] = add2(l2[e & 1], pack2(p0, p1));
                            u[e] = pack_bf16x2(p0, p1);
                        }
                        tmem_st16(hcol + 16 * c, u);
                    }
                    float l0, l1;
                    unpack2(add2(l2[0], l2[1]), l0, l1);
                    l += l0 + l1;
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                }
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[2 * t + h]);
            }
            if (!ok) break;
            ok = __all_sync(0xffffffffu, !*s_fail && mbar_wait(&o_full[t], seg & 1u));
            if (!ok) break;
            ++seg;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
            const bool done = a.shared == 0 && w.whole();
            const float inv = 1.f / l;
            const int64_t slot = a.shared > 0 ? (int64_t)w.idx + cta : 2 * cta + (w.first ? 0 : 1);
            const int64_t part_row = slot * a.part_rows + 128 * t;
            // The rows leave through this warp's share of the query tile (8 KB, free until the
            // next segment's queries come): a thread has a row, a store should have few rows.
            unsigned char *stage = s_q + t * SM::QPARTS * kPtTile;
            auto place = [&](int rk, int c) {  // 16-byte chunk c of 16 of row rk of the tile
                return reinterpret_cast<uint4 *>(stage + (c >> 3) * kPtHalf + rk * 128 + (((c & 7) ^ (rk & 7)) << 4));
            };
            const long long at = live ? (row * a.nq + head) * 128 : -1;
            const unsigned some = __ballot_sync(0xffffffffu, live);
            if (warp_live && done) {
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {
                    float v[32];
                    tmem_ld32(ocol + 32 * c, v);
                    tmem_ld_wait();
                    tmem_ld_done(v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t u[4];
#pragma unroll
                        for (int y = 0; y < 4; ++y)
                            u[y] = l != 0.f ? pack_bf16x2(v[8 * e + 2 * y] * inv, v[8 * e + 2 * y + 1] * inv) : 0u;
                        *place(r, 4 * c + e) = make_uint4(u[0], u[1], u[2], u[3]);
                    }
                }
                __syncwarp();
#pragma unroll 4
                for (int k = 0; k < 32; k += 2) {  // two rows of 256 bytes at a time
                    const int rk = k + (lane >> 4);
                    const long long o = __shfl_sync(0xffffffffu, at, rk);
                    const uint4 u = *place(32 * qd + rk, lane & 15);
                    if (o >= 0) reinterpret_cast<uint4 *>(a.o + o)[lane & 15] = u;
                }
                if (live && a.lse) a.lse[row * a.nq + head] = l != 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
            } else if (warp_live) {
#pragma unroll 1
                for (int c2 = 0; c2 < 2; ++c2) {  // 64 dims at a time
                    float v[64];
                    tmem_ld32(ocol + 64 * c2, v);
                    tmem_ld32(ocol + 64 * c2 + 32, v + 32);
                    tmem_ld_wait();
                    tmem_ld_done(v);
                    tmem_ld_done(v + 32);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        *place(r, e) = make_uint4(__float_as_uint(v[4 * e]), __float_as_uint(v[4 * e + 1]),
                                                  __float_as_uint(v[4 * e + 2]), __float_as_uint(v[4 * e + 3]));
                    __syncwarp();
                    float *po = a.part_o + (part_row + 32 * qd + (lane >> 4)) * 128 + 64 * c2;
                    uint4 u[16];
#pragma unroll
                    for (int k = 0; k < 16; ++k) u[k] = *place(32 * qd + 2 * k + (lane >> 4), lane & 15);
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (some >> (2 * k + (lane >> 4)) & 1u) reinterpret_cast<uint4 *>(po + 256 * k)[lane & 15] = u[k];
                    __syncwarp();
                }
                if (live) *reinterpret_cast<float2 *>(a.part_ml + (part_row + r) * 2) = make_float2(m, l);
            }
            __syncwarp();
            if (another) load_q(nx);
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_empty[t]);
            // the first CTA of a cut item leaves its place for the join
            if (t == 0 && r == 0 && a.cut && w.i0 == 0 && !done) {
                const int last = paged_cta_of(U, G, w.u + x.ntk - 1);
                a.cut[cta] = make_int4(x.row0, x.ntok | (w.first ? 0 : 1 << 30), w.j, last - cta + 1);
            }
            w = nx;
        } while (another);
        if (!ok) *s_fail = 1;
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    if (*s_fail && threadIdx.x == 0) {
        record_error(8u);
        const int e1 = *s_issued;
        for (int e = e1 > NST ? e1 - NST : 0; e < e1; ++e) mbar_wait(e & 1 ? &full_v[e % NST] : &full_k[e % NST], (unsigned)((e / NST) >> 1) & 1u);
    }
    __syncthreads();
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512));
    }
}

// ---- joins: a warp per row, four dimensions per lane.  A handful of loads
// ---- each, so latency is what they cost: the parts' maxima and sums are read
// ---- by a lane each, the outputs several at a time.

constexpr int kPtJoinThreads = 256;
constexpr int kPtJoinRows = kPtJoinThreads / 32;  // rows per block

// The sum over parts x < n of a row: part(x) is its place in part_ml / part_o;
// extra: one more (max, sum, outputs), or NULL.
template <typename Part>
__device__ __forceinline__ void paged_join_row(int lane, int n, const float *part_ml, const float *part_o, Part part,
                                               const float2 *extra_ml, const float4 *extra_o, int64_t row,
                                               __nv_bfloat16 *o, float *lse) {
    auto ml_of = [&](int x) { return __ldcg(reinterpret_cast<const float2 *>(part_ml) + part(x)); };
    const float2 none = make_float2(-INFINITY, 0.f);
    const float2 first = lane < n ? ml_of(lane) : none, ext = extra_ml ? __ldcg(extra_ml) : none;
    float M = fmaxf(first.x, ext.x);
    for (int x = lane + 32; x < n; x += 32) M = fmaxf(M, ml_of(x).x);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
    auto add = [&](float wt, float l, const float4 *p) {
        if (l == 0.f) return;  // nothing seen: the part's outputs may be anything (NaN keys: l is NaN)
        const float4 y = __ldcg(p + lane);
        num.x += wt * y.x;
        num.y += wt * y.y;
        num.z += wt * y.z;
        num.w += wt * y.w;
        den += wt * l;
    };
    auto weight = [&](float m) { return m == -INFINITY ? 0.f : exp2f(m - M); };
    for (int x0 = 0; x0 < n; x0 += 32) {
        const float2 ml = x0 == 0 ? first : x0 + lane < n ? ml_of(x0 + lane) : none;
        const float wt = weight(ml.x);
#pragma unroll 4
        for (int x = 0; x < min(32, n - x0); ++x)
            add(__shfl_sync(0xffffffffu, wt, x), __shfl_sync(0xffffffffu, ml.y, x),
                reinterpret_cast<const float4 *>(part_o) + part(x0 + x) * 32);
    }
    if (extra_ml) add(weight(ext.x), ext.y, extra_o);
    const float inv = 1.f / den;
    uint2 u = make_uint2(0u, 0u);
    if (den != 0.f) u = make_uint2(pack_bf16x2(num.x * inv, num.y * inv), pack_bf16x2(num.z * inv, num.w * inv));
    reinterpret_cast<uint2 *>(o + row * 128)[lane] = u;
    if (lse && lane == 0) lse[row] = den != 0.f ? (M + log2f(den)) * 0.6931471805599453f : -INFINITY;
}

// The items that were cut: block (c, k) takes rows kPtJoinRows k .. of the item whose first CTA is c.
__global__ void __launch_bounds__(kPtJoinThreads) paged_prompt_join_kernel(const __grid_constant__ PagedPromptArgs a) {
    pdl_wait();
    pdl_trigger();
    const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 cut = a.cut[c];
    if (cut.w == 0) return;
    const int ntok = cut.y & 0xffff, slot0 = 2 * c + (cut.y >> 30 & 1);
    const int rr = blockIdx.y * kPtJoinRows + warp, r = rr & 127;
    const int tok = (rr >> 7) * a.tb + r / a.g;
    if (r >= a.tb * a.g || tok >= ntok) return;
    const int64_t row = (int64_t)(cut.x + tok) * a.nq + cut.z * a.g + r % a.g;
    paged_join_row(lane, cut.w, a.part_ml, a.part_o,
                   [&](int x) { return (int64_t)(x == 0 ? slot0 : 2 * (c + x)) * a.part_rows + rr; }, nullptr, nullptr, row,
                   a.o, a.lse);
}

// For every (sequence, query head) of a batch behind a common prefix: the
// prefix's partials and what the sequence's own keys gave.
struct PagedSharedJoinArgs {
    PagedPromptArgs p;
    int G;                       // CTAs the prefix was cut into
    const float *own_o, *own_ml; // [n_seqs][nq][128], [n_seqs][nq][2]
};

__global__ void __launch_bounds__(kPtJoinThreads) paged_shared_join_kernel(const __grid_constant__ PagedSharedJoinArgs g) {
    pdl_wait();
    pdl_trigger();
    const PagedPromptArgs &a = g.p;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.ready = 0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row = (int64_t)blockIdx.x * kPtJoinRows + warp;
    if (row >= (int64_t)a.v.n_tokens * a.nq) return;
    const int b = (int)(row / a.nq), head = (int)(row % a.nq), j = head / a.g;
    const int items = pt_items(a, a.v.n_tokens), it = b / (2 * a.tb), tok = b % (2 * a.tb);
    const int rr = tok / a.tb * 128 + tok % a.tb * a.g + head % a.g;
    const int64_t NT = (a.shared + kPtKeys - 1) / kPtKeys, idx = (int64_t)j * items + it;
    const int64_t U = NT * items * a.v.nkv;
    const int cf = paged_cta_of(U, g.G, idx * NT), cl = paged_cta_of(U, g.G, idx * NT + NT - 1);
    paged_join_row(lane, cl - cf + 1, a.part_ml, a.part_o, [&](int x) { return (idx + cf + x) * a.part_rows + rr; },
                   reinterpret_cast<const float2 *>(g.own_ml) + row,
                   reinterpret_cast<const float4 *>(g.own_o) + row * 32, row, a.o, a.lse);
}

}  // namespace tpl
