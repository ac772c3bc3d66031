// Owned-head GQA attention of single tokens over a paged cache (ragged
// lengths; a sliding window with a few first tokens that stay visible).
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = 2^(x_j - m),  x_j = log2(e) q.k_j / sqrt(128),
// over the keys j of the token's sequence with j < len and (j >= lo or j <
// sinks), lo = len - window (0 without a window).  Every visible key and value
// is read once and used by the g query heads of its kv head: at most 8
// multiply-adds per byte (16 with the low parts below), so HBM is the bound.
//
// The work is cut at the device, because only the device knows the lengths:
// the visible blocks of 64 keys of every (sequence, kv head) pair are laid
// end to end, and CTA c of G takes the contiguous range [U c / G, U (c+1) / G)
// of them, so every SM streams the same bytes however ragged the batch is.
// Each CTA finds its range from a prefix sum over the sequences.  A pair that
// lies in one CTA is finished there; one that is cut leaves partials (max, sum,
// unnormalised output) and the last of its CTAs to arrive joins them in CTA
// order, so results do not depend on the timing.
//
// Per CTA: one producer warp issues the TMA copies (a lane per page part: all
// 128 dimensions of at most 64 keys of one page) into a ring of stages of 64
// keys; it looks the pages of 32 parts up at once, a batch ahead.  Two groups
// of four warps take alternate stages, 16 keys per warp, on mma.sync m16n8k16:
// the queries are carried as bf16 hi + lo parts (q is fp32: together 16 bits of
// mantissa), as is P: each is off by about 2^-16 of its value, far below the bf16
// cache and a bf16 o (a plan with fp32 outputs is limited by it).
// With g <= 8 the two parts are rows 0-7 and 8-15 of one product; with g up to
// 16 they are two products.  tcgen05 would pad the g rows to 128.
// At the end of a pair the eight warps leave their states in shared memory and
// go on; two merging warps join them, write the result and bring the queries
// of later pairs, so that short sequences do not wait on each other's ends (the
// keys of 64 sequences of 130 to 512 behind a prefix: 72 us before, 47 with
// them).
// Measured: 16 tokens at 8193 keys, 64/8 heads, 95 us (5.7 TB/s); 32 tokens with
// a window of 4096 on pages of 16, 100 us (5.2 TB/s).
//
// A page none of whose keys is visible is not read, nor is its table entry;
// keys that are not visible are masked by a select and their values replaced
// by zero, so nothing that a page holds there (stale data, NaN) is seen.
#pragma once

#include <cuda.h>

#include "tpl_attn_tma.cuh"
#include "tpl_paged.cuh"

namespace tpl {

constexpr int kPdKeys = 64;                       // keys per stage
constexpr int kPdBox = kPdKeys * 128;             // 64 keys x 64 dims, bf16: 8 KB
constexpr int kPdStage = 4 * kPdBox;              // K low and high dims, V low and high dims
constexpr int kPdMergeWarp = kAmWarps + 1;        // first merging warp, behind the producer
constexpr int kPdMergeWarps = 2;
constexpr int kPdThreads = (kPdMergeWarp + kPdMergeWarps) * 32;  // 8 consumer warps, the producer, the merging warps
// Blocks per CTA at least: fewer make more CTAs, but more joins.  With 1, 2, 4, 8 and 16: one
// token at 131 keys, 8/8 heads 8.9, 10.4, 10.4, 13.0 and 11.6 us; at 518, 32/32 13.8, 13.6,
// 12.2, 12.9 and 16.1; at 518, 64/8 13.5, 16.6, 14.8, 15.4 and 18.1; at 2001, 32/8 14.5, 12.3,
// 11.6, 13.6 and 15.8; 5 at 201, 32/32 13.4, 13.5, 13.4, 10.2 and 14.5; 8 at 1001, 64/8 20.9,
// 21.2, 21.3, 17.3 and 13.9; one at 8193, 64/8 23.7, 23.6, 23.6, 22.0 and 21.1.  No value is
// best everywhere: what decides is whether the pairs end up cut.
constexpr int kPdMinBlocks = 4;
constexpr int kPdRow = 136;                       // floats between the rows of a state: 8 rows apart in banks

template <int GM>
struct PdSmem {
    static constexpr int NS = 4;
    // a stage belongs to one group: its parity names a lap only to a reader
    // that has seen the lap before land
    static_assert(NS % kAmGroups == 0, "stages per group");
    static constexpr int SLOTS = GM == 8 ? 2 : 1;              // states of finished pairs
    static constexpr int STATE = kAmWarps * GM * kPdRow * 4;   // [8 warps][GM][kPdRow]
    static constexpr int ML = kAmWarps * GM * 8;               // [8 warps][GM](max, sum)
    static constexpr int Q = 2 * GM * 256;                     // hi rows, lo rows; two pairs
    static constexpr int JOIN = kAmWarps * GM * 4 + 2 * GM * 4;  // the merge's weights, maxima and sums
    static constexpr int BAR = 512;
    static constexpr int SCAN = (kPagedMaxSeqs + 1) * 8 + kPagedMaxSeqs * 4;
    static constexpr size_t BYTES = (size_t)NS * kPdStage + 2 * Q + SLOTS * (STATE + ML) + JOIN + BAR + SCAN;
    static_assert(BYTES <= 232448, "shared memory per block");
    static_assert(kPagedMaxCtas * GM * 3 * 4 <= STATE, "the join's tables");
};

struct PagedDecodeArgs {
    CUtensorMap tm_k, tm_v;  // 64 dims x pool rows x 2 halves, boxes of 64 x min(64, page) x 2
    PagedView v;
    const void *q;           // [n_seqs] rows
    int q_f32;
    int64_t q_ts, q_hs;
    int nq, g;
    int window, sinks;       // window 0: none
    int base;                // keys before this one are left out (a shared prefix)
    float scale_log2;
    float *part_o;           // [2 * grid][g][128]
    float *part_ml;          // [2 * grid][g][2]
    unsigned *tickets;       // [grid], by the first CTA of a cut pair
    void *o;                 // [n_seqs][nq * 128] activation type
    int o_f32;
    float *lse;              // [n_seqs][nq] or NULL
    float *own_o;            // when set (a shared prefix): unnormalised fp32 outputs [n_seqs][nq][128]
    float *own_ml;           // and (max, sum) [n_seqs][nq][2] instead of o and lse.  The kernel before this
                             // one is then the prefix's: it has waited for all that came before and passes
                             // that on by `ready`; nothing here needs it, so this one starts at once and waits
                             // for it at its end.
    const unsigned *ready;
};

// What one sequence's token sees, in keys and in blocks.
struct PdSpan {
    int len, lo, sk;   // visible: j < len && (j >= lo || j < sk)
    int nsb, fb, nblk; // blocks: 0 .. nsb-1, then fb ..
    __device__ __forceinline__ int block(int i) const { return i < nsb ? i : fb + i - nsb; }
    __device__ __forceinline__ bool sees(int j) const { return j < len && (j >= lo || j < sk); }
};

__device__ __forceinline__ PdSpan pd_span(const PagedDecodeArgs &a, int len) {
    PdSpan s;
    s.len = len;
    s.lo = a.window > 0 ? max(0, len - a.window) : 0;
    s.lo = max(s.lo, a.base);
    s.sk = min(a.sinks, s.lo);
    s.nsb = (s.sk + kPdKeys - 1) / kPdKeys;
    s.fb = max(s.lo / kPdKeys, s.nsb);
    const int lb = (int)(((int64_t)len + kPdKeys - 1) / kPdKeys);
    s.nblk = len > a.base ? s.nsb + max(0, lb - s.fb) : 0;
    return s;
}

// (sequence, kv head, block) of the units in order.
struct PdWalk {
    int b, j;
    PdSpan sp;
    __device__ __forceinline__ void open(const PagedDecodeArgs &a, const int *len, int b_) {
        b = b_;
        sp = pd_span(a, len[b]);
    }
    // the next pair
    __device__ __forceinline__ void next(const PagedDecodeArgs &a, const long long *start, const int *len) {
        if (++j == a.v.nkv) {
            j = 0;
            do ++b;
            while (start[b + 1] == start[b]);
            open(a, len, b);
        }
    }
};

template <int GM>
__global__ void __launch_bounds__(kPdThreads, 1) paged_decode_kernel(const __grid_constant__ PagedDecodeArgs a) {
    constexpr int D = 128;
    using SM = PdSmem<GM>;
    constexpr int NS = SM::NS, NB = SM::SLOTS;
    constexpr int RPT = GM / 8;  // rows (heads) per thread
    extern __shared__ __align__(1024) unsigned char pd_raw[];
    unsigned char *sm = pd_raw;
    if (smem_u32(sm) & 1023u) {  // (the whole grid: the swizzled stages need 1 KB alignment)
        if (threadIdx.x == 0) record_error(8u);
        pdl_wait();
        return;
    }
    unsigned char *s_q = sm + NS * kPdStage;                                   // [2][hi, lo][GM][256 B], swizzled
    float *s_o = reinterpret_cast<float *>(s_q + 2 * SM::Q);                   // [NB][8 warps][GM][kPdRow]
    float *s_ml = s_o + NB * SM::STATE / 4;                                    // [NB][8 warps][GM][2]
    float *s_wt = s_ml + NB * SM::ML / 4;                                      // [8 warps][GM]
    float *s_M = s_wt + kAmWarps * GM, *s_den = s_M + GM;
    uint64_t *full = reinterpret_cast<uint64_t *>(s_den + GM);
    uint64_t *empty = full + NS;
    uint64_t *q_full = empty + NS;     // [2]
    uint64_t *st_full = q_full + 2;    // [NB]
    uint64_t *st_empty = st_full + NB; // [NB]
    volatile int *s_flag = reinterpret_cast<volatile int *>(st_empty + NB);  // fail, last, issued
    long long *s_warp = reinterpret_cast<long long *>(st_empty + NB + 2);    // [warps]
    static_assert((2 * NS + 2 + 2 * NB + 2 + kPdThreads / 32) * 8 <= SM::BAR, "barrier area");
    long long *s_start = reinterpret_cast<long long *>(reinterpret_cast<unsigned char *>(full) + SM::BAR);  // [n_seqs + 1]
    int *s_len = reinterpret_cast<int *>(s_start + kPagedMaxSeqs + 1);  // [n_seqs]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    const PagedView &v = a.v;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kAmGroupWarps);
        }
        for (int s = 0; s < 2; ++s) mbar_init(&q_full[s], kPdMergeWarps);
        for (int s = 0; s < NB; ++s) {
            mbar_init(&st_full[s], kAmWarps);
            mbar_init(&st_empty[s], kPdMergeWarps);
        }
        s_flag[0] = 0;
        s_flag[1] = 0;
        s_flag[2] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (!a.own_o || !pdl_passed_on(a.ready)) pdl_wait();
    pdl_trigger();

    // ---- prefix sums of the sequences' blocks (all kv heads) ----
    {
        constexpr int PT = (kPagedMaxSeqs + kPdThreads - 1) / kPdThreads;
        const int per = (v.n_seqs + kPdThreads - 1) / kPdThreads;
        long long mine[PT], sum = 0;
#pragma unroll
        for (int x = 0; x < PT; ++x) {
            const int b = threadIdx.x * per + x;
            mine[x] = 0;
            if (x < per && b < v.n_seqs) {
                const int len = paged_len(v, b);
                s_len[b] = len;
                mine[x] = (long long)pd_span(a, len).nblk * v.nkv;
            }
            sum += mine[x];
        }
        long long inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += t;
        }
        if (lane == 31) s_warp[warp] = inc;
        __syncthreads();
        long long at = inc - sum;
        for (int w = 0; w < warp; ++w) at += s_warp[w];
#pragma unroll
        for (int x = 0; x < PT; ++x) {
            const int b = threadIdx.x * per + x;
            if (x < per && b < v.n_seqs) {
                s_start[b] = at;
                at += mine[x];
                if (b == v.n_seqs - 1) s_start[v.n_seqs] = at;
            }
        }
        __syncthreads();
    }
    const int64_t U = s_start[v.n_seqs];
    const int G = (int)min((int64_t)gridDim.x, max((int64_t)1, (U + kPdMinBlocks - 1) / kPdMinBlocks));

    // sequences that see nothing: zeros (no keys: an empty softmax)
    for (int b = cta; b < v.n_seqs; b += gridDim.x) {
        if (s_start[b + 1] != s_start[b]) continue;
        for (int x = threadIdx.x; x < a.nq * D; x += kPdThreads)
            if (!a.own_o) store_act(a.o, a.o_f32, (int64_t)b * a.nq * D + x, 0.f);
        for (int x = threadIdx.x; x < a.nq; x += kPdThreads) {
            if (a.own_o) {
                a.own_ml[((int64_t)b * a.nq + x) * 2] = -INFINITY;
                a.own_ml[((int64_t)b * a.nq + x) * 2 + 1] = 0.f;
            } else if (a.lse) {
                a.lse[(int64_t)b * a.nq + x] = -INFINITY;
            }
        }
    }
    if (cta >= G || U == 0) {  // the whole CTA: nothing in flight
        if (a.own_o) pdl_wait();
        return;
    }

    const int64_t u0 = paged_cut(U, G, cta), u1 = paged_cut(U, G, cta + 1);
    const int n = (int)(u1 - u0);
    // the sequence of unit u: the last one that begins at or before it
    auto seq_of = [&](int64_t u) {
        int l = 0, r = v.n_seqs - 1;
        while (l < r) {
            const int mid = (l + r + 1) >> 1;
            if (s_start[mid] <= u) l = mid;
            else r = mid - 1;
        }
        return l;
    };
    const int box_shift = min(v.page_shift, 6);  // rows per copy

    if (warp == kAmWarps) {
        // ---- producer: lane = (K or V, page part) ----
        const uint64_t kvpol = evict_first_policy();
        const int nsub = kPdKeys >> box_shift;  // parts of a block: 1, 2 or 4
        const int batch = 32 / nsub;            // blocks per lookup
        const int kv = lane / nsub, sub = lane % nsub;
        // the pool row of part lane % nsub of unit i0 + lane / nsub, -1 when no key of it is seen
        auto lookup = [&](int i0) {
            const int i = min(i0 + lane / nsub, n - 1);
            const int64_t u = u0 + i;
            PdWalk w;
            w.open(a, s_len, seq_of(u));
            const int64_t rel = u - s_start[w.b];
            w.j = (int)paged_div(rel, w.sp.nblk);
            const int key = w.sp.block((int)(rel - (int64_t)w.j * w.sp.nblk)) * kPdKeys + ((lane % nsub) << box_shift);
            const bool want = i0 + lane / nsub < n && key < w.sp.len && (key + (1 << box_shift) > w.sp.lo || key < w.sp.sk);
            if (!want) return -1;
            const int64_t r = paged_row(v, w.b, key >> v.page_shift, w.j);
            return r < 0 ? 0 : (int)r + (key & ((1 << v.page_shift) - 1));
        };
        int ahead = lookup(0);
        bool ok = true;
        int i = 0;
        for (int ib = 0; ok && ib < n; ib += batch) {
            const int rows = ahead;
            if (ib + batch < n) ahead = lookup(ib + batch);
            for (; i < min(ib + batch, n); ++i) {
                const int s = i % NS;
                const int row = __shfl_sync(0xffffffffu, rows, (i - ib) * nsub + sub);
                const bool want = kv < 2 && row >= 0;
                const unsigned bytes = (unsigned)__popc(__ballot_sync(0xffffffffu, want)) << (box_shift + 8);
                if (lane == 0) {
                    ok = !s_flag[0] && mbar_wait(&empty[s], ((unsigned)(i / NS) & 1u) ^ 1u);
                    if (ok) mbar_expect_tx(&full[s], bytes);
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0);
                if (!ok) break;
                if (want)
                    tma_load_3d_hint(sm + s * kPdStage + kv * 2 * kPdBox + (sub << (box_shift + 8)),
                                     kv ? &a.tm_v : &a.tm_k, 0, row, 0, &full[s], kvpol);
            }
        }
        if (!ok) s_flag[0] = 1;
        if (lane == 0) s_flag[2] = i;
    } else if (warp < kAmWarps) {
        // ---- consumers: group grp takes the stages i with i % kAmGroups == grp ----
        const int gid = lane >> 2, c = lane & 3;
        const int grp = warp / kAmGroupWarps, wl = warp % kAmGroupWarps;
        bool dead = false;  // after a timeout the warps walk on without waiting, so that every barrier still meets
        // this warp's 16 keys of a stage: their rows in the part's box, the two halves of the dims
        const unsigned half_bytes = 1u << (box_shift + 7);
        const int row_in = (16 * wl) & ((1 << box_shift) - 1);
        const unsigned part_off = (unsigned)((16 * wl) >> box_shift) * 2 * half_bytes;
        PdWalk w;
        w.open(a, s_len, seq_of(u0));
        int64_t pair_start = s_start[w.b];
        {
            const int64_t rel = u0 - pair_start;
            w.j = (int)paged_div(rel, w.sp.nblk);
            pair_start += (int64_t)w.j * w.sp.nblk;
        }
        int i = 0;
        for (int seg = 0; i < n; ++seg) {
            // one segment: the blocks of one pair
            const PdSpan &sp = w.sp;
            const int64_t pair_end = pair_start + sp.nblk;
            const int first = (int)(u0 + i - pair_start);
            const int seg_n = (int)(min(u1, pair_end) - (u0 + i));
            // q fragments of the hi parts (GM == 8: rows 8-15 are the lo parts)
            if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(&q_full[seg & 1], (unsigned)(seg >> 1) & 1u));
            const unsigned char *q = s_q + (seg & 1) * SM::Q;
            const int q_row = (lane & 7) + ((lane >> 3 & 1) << 3), q_chunk = lane >> 4;
            auto q_frag = [&](int part, int ks, uint32_t (&f)[4]) {
                const int row = 16 * part + q_row;
                ldsm_x4(q + row * 256 + (((2 * ks + q_chunk) ^ (row & 7)) << 4), f[0], f[1], f[2], f[3]);
            };
            uint32_t qf[8][4];
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) q_frag(0, ks, qf[ks]);
            float o[16][4];
#pragma unroll
            for (int t = 0; t < 16; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
            float m[RPT], l[RPT];
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                m[r] = -INFINITY;
                l[r] = 0.f;
            }
            for (int e = 0; e < seg_n; ++e, ++i) {
                if (i % kAmGroups != grp) continue;
                const int s = i % NS;
                if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(&full[s], (unsigned)(i / NS) & 1u));
                const int kb = sp.block(first + e) * kPdKeys + 16 * wl;  // this warp's 16 keys
                if (!dead && kb < sp.len && (kb + 16 > sp.lo || kb < sp.sk)) {
                    const unsigned char *st = sm + s * kPdStage + part_off;
                    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
                    {
                        // even and odd steps add up apart: half the chain of dependent products
                        float t0[4] = {0.f, 0.f, 0.f, 0.f}, t1[4] = {0.f, 0.f, 0.f, 0.f};
                        const int row = row_in + (lane & 7) + ((lane >> 4) << 3);
                        const int half = (lane >> 3) & 1;
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            uint32_t b0_, b1_, b2_, b3_;
                            ldsm_x4(st + (ks >> 2) * half_bytes + am_swz(row, 2 * (ks & 3) + half), b0_, b1_, b2_, b3_);
                            float(&y0)[4] = ks & 1 ? t0 : s0, (&y1)[4] = ks & 1 ? t1 : s1;
                            mma_bf16_16816(y0, qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b0_, b1_);
                            mma_bf16_16816(y1, qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b2_, b3_);
                            if (RPT == 2) {
                                uint32_t ql[4];
                                q_frag(1, ks, ql);
                                mma_bf16_16816(y0, ql[0], ql[1], ql[2], ql[3], b0_, b1_);
                                mma_bf16_16816(y1, ql[0], ql[1], ql[2], ql[3], b2_, b3_);
                            }
                        }
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            s0[x] += t0[x];
                            s1[x] += t1[x];
                        }
                    }
                    // this thread's keys: kb + 2c, +1, +8, +9
                    const int kk = kb + 2 * c;
                    const bool v0 = sp.sees(kk), v1 = sp.sees(kk + 1), v2 = sp.sees(kk + 8), v3 = sp.sees(kk + 9);
                    const uint32_t keep_a = (v0 ? 0xffffu : 0u) | (v1 ? 0xffff0000u : 0u);
                    const uint32_t keep_b = (v2 ? 0xffffu : 0u) | (v3 ? 0xffff0000u : 0u);
                    uint32_t ph[RPT][2], pl[RPT][2];
#pragma unroll
                    for (int r = 0; r < RPT; ++r) {
                        float x0, x1, x2, x3;
                        if (RPT == 1) {
                            x0 = s0[0] + s0[2];
                            x1 = s0[1] + s0[3];
                            x2 = s1[0] + s1[2];
                            x3 = s1[1] + s1[3];
                        } else {
                            x0 = s0[2 * r];
                            x1 = s0[2 * r + 1];
                            x2 = s1[2 * r];
                            x3 = s1[2 * r + 1];
                        }
                        x0 = v0 ? x0 * a.scale_log2 : -INFINITY;
                        x1 = v1 ? x1 * a.scale_log2 : -INFINITY;
                        x2 = v2 ? x2 * a.scale_log2 : -INFINITY;
                        x3 = v3 ? x3 * a.scale_log2 : -INFINITY;
                        float mx = fmaxf(fmaxf(x0, x1), fmaxf(x2, x3));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                        // one of the 16 keys is visible, so mx is a logit (which may have
                        // fallen below fp32's range).  Raise the running maximum only past
                        // the margin: until then p <= 2^kAmLazy.
                        if (mx > m[r] + kAmLazy) {
                            const float alpha = exp2f(m[r] - mx);  // 0 on the first step (m = -inf)
                            m[r] = mx;
                            l[r] *= alpha;
#pragma unroll
                            for (int t = 0; t < 16; ++t) {
                                o[t][2 * r] *= alpha;
                                o[t][2 * r + 1] *= alpha;
                                if (RPT == 1) {
                                    o[t][2] *= alpha;
                                    o[t][3] *= alpha;
                                }
                            }
                        }
                        const float sub = m[r] == -INFINITY ? 0.f : m[r];  // only logits of -inf so far: 2^-inf each
                        const float p0 = ex2(x0 - sub), p1 = ex2(x1 - sub), p2 = ex2(x2 - sub), p3 = ex2(x3 - sub);
                        l[r] += (p0 + p1) + (p2 + p3);
                        ph[r][0] = pack_bf16x2(p0, p1);
                        ph[r][1] = pack_bf16x2(p2, p3);
                        pl[r][0] = pack_bf16x2(p0 - bf16lo(ph[r][0]), p1 - bf16hi(ph[r][0]));
                        pl[r][1] = pack_bf16x2(p2 - bf16lo(ph[r][1]), p3 - bf16hi(ph[r][1]));
                    }
                    {
                        const int row = row_in + (lane & 7) + (((lane >> 3) & 1) << 3);
                        const int half = lane >> 4;
#pragma unroll
                        for (int n2 = 0; n2 < 8; ++n2) {
                            uint32_t w0, w1, w2, w3;
                            ldsm_x4_t(st + 2 * kPdBox + (n2 >> 2) * half_bytes + am_swz(row, 2 * (n2 & 3) + half), w0, w1, w2,
                                      w3);
                            w0 &= keep_a;
                            w1 &= keep_b;
                            w2 &= keep_a;
                            w3 &= keep_b;
                            if (RPT == 1) {
                                mma_bf16_16816(o[2 * n2], ph[0][0], pl[0][0], ph[0][1], pl[0][1], w0, w1);
                                mma_bf16_16816(o[2 * n2 + 1], ph[0][0], pl[0][0], ph[0][1], pl[0][1], w2, w3);
                            } else {
                                constexpr int R1 = RPT - 1;
                                mma_bf16_16816(o[2 * n2], ph[0][0], ph[R1][0], ph[0][1], ph[R1][1], w0, w1);
                                mma_bf16_16816(o[2 * n2], pl[0][0], pl[R1][0], pl[0][1], pl[R1][1], w0, w1);
                                mma_bf16_16816(o[2 * n2 + 1], ph[0][0], ph[R1][0], ph[0][1], ph[R1][1], w2, w3);
                                mma_bf16_16816(o[2 * n2 + 1], pl[0][0], pl[R1][0], pl[0][1], pl[R1][1], w2, w3);
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[s]);
            }
            // ---- leave the state to the merging warps ----
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            }
            const int slot = seg % NB;
            if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(&st_empty[slot], ((unsigned)(seg / NB) & 1u) ^ 1u));
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const int hd = gid + 8 * r;
                if (hd < a.g) {
                    float *p = s_o + slot * (SM::STATE / 4) + (warp * GM + hd) * kPdRow + 2 * c;
#pragma unroll
                    for (int t = 0; t < 16; ++t)  // (GM == 8: rows gid + 8 held the P_lo . V part of the same head)
                        *reinterpret_cast<float2 *>(p + 8 * t) =
                            RPT == 1 ? make_float2(o[t][0] + o[t][2], o[t][1] + o[t][3])
                                     : make_float2(o[t][2 * r], o[t][2 * r + 1]);
                    if (c == 0)
                        *reinterpret_cast<float2 *>(s_ml + slot * (SM::ML / 4) + (warp * GM + hd) * 2) = make_float2(m[r], l[r]);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&st_full[slot]);
            pair_start = pair_end;
            if (i < n) w.next(a, s_start, s_len);
        }
        if (dead) s_flag[0] = 1;
    } else {
        // ---- merging warps: every other head each, a lane four dimensions ----
        const int tid = threadIdx.x - kPdMergeWarp * 32, mw = warp - kPdMergeWarp;
        auto meet = [] { asm volatile("bar.sync 2, %0;" ::"n"(kPdMergeWarps * 32) : "memory"); };
        bool dead = false;
        PdWalk w, ahead;
        w.open(a, s_len, seq_of(u0));
        int64_t pair_start = s_start[w.b];
        {
            const int64_t rel = u0 - pair_start;
            w.j = (int)paged_div(rel, w.sp.nblk);
            pair_start += (int64_t)w.j * w.sp.nblk;
        }
        // The queries of the segments to come: loaded three segments ahead, stored (rows of hi
        // parts, then of lo parts) two ahead, when the consumers are done with the buffer.
        ahead = w;
        int64_t ahead_at = pair_start;  // where its pair begins; at or behind u1: no such segment
        int staged = 0;
        bool held = false;
        uint4 raw[2 * RPT][2];
        auto load_q = [&]() {
            held = ahead_at < u1;
            if (!held) return;
#pragma unroll
            for (int r = 0; r < 2 * RPT; ++r) {
                const int hd = tid / 16 + 4 * r, ch = tid % 16;  // 8 dims
                raw[r][0] = raw[r][1] = make_uint4(0, 0, 0, 0);
                if (hd < a.g) {
                    const int64_t off = ahead.b * a.q_ts + (ahead.j * a.g + hd) * a.q_hs + 8 * ch;
                    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const char *>(a.q) + off * (a.q_f32 ? 4 : 2));
                    raw[r][0] = p[0];
                    if (a.q_f32) raw[r][1] = p[1];
                }
            }
            ahead_at += ahead.sp.nblk;
            if (ahead_at < u1) ahead.next(a, s_start, s_len);
        };
        auto store_q = [&]() {
            if (!held) return;
            unsigned char *q = s_q + (staged & 1) * SM::Q;
#pragma unroll
            for (int r = 0; r < 2 * RPT; ++r) {
                const int hd = tid / 16 + 4 * r, ch = tid % 16;
                uint32_t h[4], lo[4];
                const uint32_t y[8] = {raw[r][0].x, raw[r][0].y, raw[r][0].z, raw[r][0].w,
                                       raw[r][1].x, raw[r][1].y, raw[r][1].z, raw[r][1].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (a.q_f32) {
                        const float f0 = __uint_as_float(y[2 * e]), f1 = __uint_as_float(y[2 * e + 1]);
                        h[e] = pack_bf16x2(f0, f1);
                        lo[e] = pack_bf16x2(f0 - bf16lo(h[e]), f1 - bf16hi(h[e]));
                    } else {
                        h[e] = y[e];
                        lo[e] = 0u;
                    }
                }
                const int at = (ch ^ (hd & 7)) << 4;
                *reinterpret_cast<uint4 *>(q + hd * 256 + at) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4 *>(q + (GM + hd) * 256 + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&q_full[staged & 1]);
            ++staged;
        };
        load_q();
        store_q();
        load_q();
        store_q();
        load_q();
        for (int seg = 0; pair_start < u1; ++seg) {
            const int64_t pair_end = pair_start + w.sp.nblk;
            const int slot = seg % NB;
            const float *so = s_o + slot * (SM::STATE / 4), *sml = s_ml + slot * (SM::ML / 4);
            if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(&st_full[slot], (unsigned)(seg / NB) & 1u));
            store_q();  // (into the buffer of this segment: every consumer is done with it)
            load_q();
            // weights of the eight states of a head: eight lanes side by side
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                const int x = tid & 7, hd = (tid >> 3) + 8 * r;
                const float2 ml = hd < a.g ? *reinterpret_cast<const float2 *>(sml + (x * GM + hd) * 2) : make_float2(-INFINITY, 0.f);
                float M = ml.x;
#pragma unroll
                for (int k = 4; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, k));
                const float wt = ml.x == -INFINITY ? 0.f : exp2f(ml.x - M);
                float den = wt * ml.y;
#pragma unroll
                for (int k = 4; k > 0; k >>= 1) den += __shfl_xor_sync(0xffffffffu, den, k);
                if (hd < a.g) {
                    s_wt[x * GM + hd] = wt;
                    if (x == 0) {
                        s_M[hd] = M;
                        s_den[hd] = den;
                    }
                }
            }
            meet();
            const bool whole = pair_start >= u0 && pair_end <= u1;
            const int cf = whole ? cta : paged_cta_of(U, G, pair_start);
            auto emit = [&](int hrow, const float4 &num, float M, float den) {
                const int64_t row = (int64_t)w.b * a.nq + w.j * a.g + hrow;
                if (a.own_o) {
                    reinterpret_cast<float4 *>(a.own_o + row * D)[lane] = num;
                    if (lane == 0) *reinterpret_cast<float2 *>(a.own_ml + row * 2) = make_float2(M, den);
                } else {
                    const float inv = den != 0.f ? 1.f / den : 0.f;  // 0: only logits of -inf
                    if (a.o_f32)
                        reinterpret_cast<float4 *>(static_cast<float *>(a.o) + row * D)[lane] =
                            make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
                    else
                        reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.o) + row * D)[lane] =
                            make_uint2(pack_bf16x2(num.x * inv, num.y * inv), pack_bf16x2(num.z * inv, num.w * inv));
                    if (a.lse && lane == 0) a.lse[row] = (M + log2f(den)) * 0.6931471805599453f;
                }
            };
            auto add = [](float4 &num, float wt, const float4 &y) {
                num.x += wt * y.x;
                num.y += wt * y.y;
                num.z += wt * y.z;
                num.w += wt * y.w;
            };
            const int64_t part = 2 * cta + (pair_start > u0 ? 1 : 0);
#pragma unroll 2
            for (int hrow = mw; hrow < a.g; hrow += kPdMergeWarps) {
                float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int x = 0; x < kAmWarps; ++x)
                    add(num, s_wt[x * GM + hrow], reinterpret_cast<const float4 *>(so + (x * GM + hrow) * kPdRow)[lane]);
                if (whole) {
                    emit(hrow, num, s_M[hrow], s_den[hrow]);
                } else {
                    reinterpret_cast<float4 *>(a.part_o + (part * a.g + hrow) * D)[lane] = num;
                    if (lane == 0)
                        *reinterpret_cast<float2 *>(a.part_ml + (part * a.g + hrow) * 2) = make_float2(s_M[hrow], s_den[hrow]);
                }
            }
            if (!whole) {
                const int n_p = paged_cta_of(U, G, pair_end - 1) - cf + 1;
                __threadfence();
                meet();
                if (tid == 0) {
                    const unsigned prev = atomicAdd(&a.tickets[cf], 1u);
                    s_flag[1] = prev == (unsigned)(n_p - 1);
                    if (prev >= (unsigned)n_p) record_error(2u);
                }
                meet();
                if (s_flag[1]) {
                    // ---- the last CTA of the pair: partials in CTA order.  The state of this
                    //      segment has been read, so its slot holds the tables. ----
                    __threadfence();
                    float *s_mlp = s_o + slot * (SM::STATE / 4);  // [n_p][g][2]
                    float *s_w = s_mlp + 2 * GM * kPagedMaxCtas;  // [n_p][GM]
                    // CTA cf's part of the pair is its second segment when its range begins before the pair
                    const int part0 = 2 * cf + (paged_cut(U, G, cf) < pair_start ? 1 : 0);
                    auto part_of = [&](int x) { return x == 0 ? part0 : 2 * (cf + x); };
                    for (int x = tid; x < n_p * a.g; x += kPdMergeWarps * 32) {
                        const float2 ml = __ldcg(reinterpret_cast<const float2 *>(a.part_ml) +
                                                 (int64_t)part_of(x / a.g) * a.g + x % a.g);
                        s_mlp[2 * x] = ml.x;
                        s_mlp[2 * x + 1] = ml.y;
                    }
                    meet();
                    if (tid < a.g) {
                        float M = -INFINITY;
                        for (int x = 0; x < n_p; ++x) M = fmaxf(M, s_mlp[(x * a.g + tid) * 2]);
                        float den = 0.f;
                        for (int x = 0; x < n_p; ++x) {
                            const float mi = s_mlp[(x * a.g + tid) * 2];
                            const float wt = mi == -INFINITY ? 0.f : exp2f(mi - M);
                            s_w[x * GM + tid] = wt;
                            den += wt * s_mlp[(x * a.g + tid) * 2 + 1];
                        }
                        s_M[tid] = M;
                        s_den[tid] = den;
                    }
                    meet();
#pragma unroll 2
                    for (int hrow = mw; hrow < a.g; hrow += kPdMergeWarps) {
                        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                        for (int x = 0; x < n_p; ++x)
                            add(num, s_w[x * GM + hrow],
                                __ldcg(reinterpret_cast<const float4 *>(a.part_o + ((int64_t)part_of(x) * a.g + hrow) * D) + lane));
                        emit(hrow, num, s_M[hrow], s_den[hrow]);
                    }
                    if (tid == 0) atomicExch(&a.tickets[cf], 0u);
                }
            }
            meet();  // everyone has read the weights and the state
            if (lane == 0) mbar_arrive(&st_empty[slot]);
            pair_start = pair_end;
            if (pair_start < u1) w.next(a, s_start, s_len);
        }
        if (dead) s_flag[0] = 1;
    }
    __syncthreads();
    if (s_flag[0] && threadIdx.x == 0) {
        record_error(8u);
        // wait (bounded) for the copies still in flight before the CTA exits
        const int issued = s_flag[2];
        for (int x = issued - NS > 0 ? issued - NS : 0; x < issued; ++x)
            mbar_wait(&full[x % NS], (unsigned)(x / NS) & 1u);
    }
    if (a.own_o) pdl_wait();
}

}  // namespace tpl
