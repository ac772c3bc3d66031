// Owned-head GQA attention of single tokens over a paged cache (ragged
// lengths; a sliding window with a few first tokens that stay visible).
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = 2^(x_j - m),  x_j = log2(e) q.k_j / sqrt(128),
// over the keys j of the token's sequence with j < len and (j >= lo or j <
// sinks), lo = len - window (0 without a window).  Every visible key and value
// is read once and used by the g query heads of its kv head: at most 16
// multiply-adds per byte, so HBM is the bound.
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
// Per CTA one warp issues the TMA copies (a lane per page part: 64 dimensions
// of at most 64 keys of one page) into a ring of stages of 64 keys; two groups
// of four warps take alternate stages, 16 keys per warp, on mma.sync m16n8k16:
// the queries are carried as bf16 hi + lo parts (q is fp32: together 16 bits of
// mantissa), as is P, so the bf16 cache is the only rounding of the products.
// With g <= 8 the two parts are rows 0-7 and 8-15 of one product; with g up to
// 16 they are two products.  tcgen05 would pad the g rows to 128.
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
constexpr int kPdThreads = kAmThreads;            // 8 consumer warps and the producer
constexpr int kPdMinBlocks = 2;                   // blocks per CTA at least

template <int GM>
struct PdSmem {
    static constexpr int NS = GM == 8 ? 6 : 4;
    // a stage belongs to one group: its parity names a lap only to a reader
    // that has seen the lap before land
    static_assert(NS % kAmGroups == 0, "stages per group");
    static constexpr int MERGE = kAmGroupWarps * GM * 128 * 4;
    static constexpr int BAR = 3072;
    static constexpr int SCAN = (kPagedMaxSeqs + 1) * 8;
    static constexpr size_t BYTES = (size_t)NS * kPdStage + MERGE + BAR + SCAN + 1024;
    static_assert(BYTES <= 232448, "shared memory per block");
    static_assert(kPagedMaxCtas * GM * 3 * 4 <= MERGE, "the join's tables");
};

struct PagedDecodeArgs {
    CUtensorMap tm_k, tm_v;  // pool rows x 128, boxes of 64 dims x min(64, page) rows
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
    float *own_ml;           // and (max, sum) [n_seqs][nq][2] instead of o and lse
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

template <int GM>
__global__ void __launch_bounds__(kPdThreads, 1) paged_decode_kernel(const __grid_constant__ PagedDecodeArgs a) {
    constexpr int D = 128;
    using SM = PdSmem<GM>;
    constexpr int NS = SM::NS;
    constexpr int RPT = GM / 8;  // rows (heads) per thread
    extern __shared__ __align__(1024) unsigned char pd_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>(((uintptr_t)pd_raw + 1023) & ~(uintptr_t)1023);
    float *s_o = reinterpret_cast<float *>(sm + NS * kPdStage);  // [4 warps][GM][128]
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + NS * kPdStage + SM::MERGE);
    uint64_t *empty = full + NS;
    float *s_ml = reinterpret_cast<float *>(empty + NS);  // [4 warps][GM][2]
    float *s_misc = s_ml + kAmGroupWarps * GM * 2;        // M[GM], den[GM]
    long long *s_warp = reinterpret_cast<long long *>(s_misc + 2 * GM);  // [warps]
    volatile int *s_flag = reinterpret_cast<volatile int *>(s_warp + 16);  // fail, last, issued
    static_assert(2 * NS * 8 + (kAmGroupWarps * GM * 2 + 2 * GM) * 4 + 16 * 8 + 16 <= SM::BAR, "barrier area");
    long long *s_start = reinterpret_cast<long long *>(sm + NS * kPdStage + SM::MERGE + SM::BAR);  // [n_seqs + 1]

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int cta = blockIdx.x;
    const PagedView &v = a.v;
    if (threadIdx.x == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kAmGroupWarps);
        }
        s_flag[0] = 0;
        s_flag[1] = 0;
        s_flag[2] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    pdl_trigger();

    // ---- prefix sums of the sequences' blocks (all kv heads) ----
    {
        constexpr int PT = (kPagedMaxSeqs + kPdThreads - 1) / kPdThreads;
        const int per = (v.n_seqs + kPdThreads - 1) / kPdThreads;
        long long mine[PT], sum = 0;
#pragma unroll
        for (int x = 0; x < PT; ++x) {
            const int b = threadIdx.x * per + x;
            mine[x] = x < per && b < v.n_seqs ? (long long)pd_span(a, paged_len(v, b)).nblk * v.nkv : 0;
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
    if (cta >= G || U == 0) return;  // the whole CTA: nothing in flight

    const int64_t u0 = am_start(U, G, cta), u1 = am_start(U, G, cta + 1);
    const int n = (int)(u1 - u0);
    int b0;  // the sequence of unit u0
    {
        int l = 0, r = v.n_seqs - 1;  // the last b with s_start[b] <= u0 that is not empty
        while (l < r) {
            const int mid = (l + r + 1) >> 1;
            if (s_start[mid] <= u0) l = mid;
            else r = mid - 1;
        }
        b0 = l;
    }
    const int box_shift = min(v.page_shift, 6);  // rows per copy

    if (warp == kAmWarps) {
        // ---- producer: lane = (part, page part) ----
        const uint64_t kvpol = evict_first_policy();
        const int nsub = kPdKeys >> box_shift;  // copies per part
        const int part = lane / nsub, sub = lane % nsub;
        const bool active = part < 4;
        int b = b0;
        PdSpan sp = pd_span(a, paged_len(v, b));
        int64_t rel = u0 - s_start[b];
        int j = (int)(rel / sp.nblk), blk = (int)(rel % sp.nblk);
        // this lane's copy of the current unit: its key, whether any of it is visible, its pool row
        auto place = [&](bool &want, int &row) {
            const int key = sp.block(blk) * kPdKeys + (sub << box_shift);
            const int end = key + (1 << box_shift);
            want = active && key < sp.len && (end > sp.lo || key < sp.sk);
            row = 0;
            if (want) {
                const int64_t r = paged_row(v, b, key >> v.page_shift, j);
                row = r < 0 ? 0 : (int)r + (key & ((1 << v.page_shift) - 1));
            }
        };
        bool want;
        int row;
        place(want, row);
        int i = 0;
        for (; i < n; ++i) {
            const int s = i % NS;
            bool ok = true;
            if (lane == 0 && i >= NS) ok = !s_flag[0] && mbar_wait(&empty[s], ((unsigned)(i / NS) & 1u) ^ 1u);
            if (!__all_sync(0xffffffffu, ok)) {
                s_flag[0] = 1;
                break;
            }
            const unsigned ballot = __ballot_sync(0xffffffffu, want);
            if (lane == 0) mbar_expect_tx(&full[s], (unsigned)__popc(ballot) << (box_shift + 7));
            __syncwarp();
            if (want)
                tma_load_2d_hint(sm + s * kPdStage + part * kPdBox + (sub << (box_shift + 7)),
                                 part < 2 ? &a.tm_k : &a.tm_v, 64 * (part & 1), row, &full[s], kvpol);
            if (i + 1 < n) {  // the next unit's page is looked up while this one's copies fly
                if (++blk == sp.nblk) {
                    blk = 0;
                    if (++j == v.nkv) {
                        j = 0;
                        do ++b;
                        while (s_start[b + 1] == s_start[b]);
                        sp = pd_span(a, paged_len(v, b));
                    }
                }
                place(want, row);
            }
        }
        if (lane == 0) s_flag[2] = i;
    } else {
        // ---- consumers: group grp takes the stages i with i % kAmGroups == grp ----
        const int gid = lane >> 2, c = lane & 3;
        const int grp = warp / kAmGroupWarps, wl = warp % kAmGroupWarps;
        const int tid = threadIdx.x;  // group 0: 0..127, one head dimension each in the merge
        bool dead = false;
        int i = 0;
        int b = b0;
        PdSpan sp = pd_span(a, paged_len(v, b));
        int64_t pair_start = s_start[b];
        int j = 0;
        {
            const int64_t rel = u0 - pair_start;
            j = (int)(rel / sp.nblk);
            pair_start += (int64_t)j * sp.nblk;
        }
        while (i < n) {
            // one segment: the blocks of one pair
            const int64_t pair_end = pair_start + sp.nblk;
            const int first = (int)(u0 + i - pair_start);
            const int seg_n = (int)(min(u1, pair_end) - (u0 + i));
            // q fragments: row r = head, dims 16 ks + 2c (+1, +8, +9); hi and lo parts
            uint32_t qf[8][4], ql[RPT == 2 ? 8 : 1][4];
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    const int hd = gid + 8 * r;
                    float2 u = make_float2(0.f, 0.f), w = u;
                    if (hd < a.g) {
                        const int64_t off = b * a.q_ts + (j * a.g + hd) * a.q_hs + 16 * ks + 2 * c;
                        if (a.q_f32) {
                            const float *qp = static_cast<const float *>(a.q) + off;
                            u = *reinterpret_cast<const float2 *>(qp);
                            w = *reinterpret_cast<const float2 *>(qp + 8);
                        } else {
                            const __nv_bfloat16 *qp = static_cast<const __nv_bfloat16 *>(a.q) + off;
                            const uint32_t x = *reinterpret_cast<const uint32_t *>(qp);
                            const uint32_t y = *reinterpret_cast<const uint32_t *>(qp + 8);
                            u = make_float2(bf16lo(x), bf16hi(x));
                            w = make_float2(bf16lo(y), bf16hi(y));
                        }
                    }
                    const uint32_t h0 = pack_bf16x2(u.x, u.y), h2 = pack_bf16x2(w.x, w.y);
                    const uint32_t l0 = pack_bf16x2(u.x - bf16lo(h0), u.y - bf16hi(h0));
                    const uint32_t l2 = pack_bf16x2(w.x - bf16lo(h2), w.y - bf16hi(h2));
                    if (RPT == 1) {
                        qf[ks][0] = h0;
                        qf[ks][1] = l0;
                        qf[ks][2] = h2;
                        qf[ks][3] = l2;
                    } else {
                        qf[ks][r] = h0;
                        qf[ks][2 + r] = h2;
                        ql[RPT == 2 ? ks : 0][r] = l0;
                        ql[RPT == 2 ? ks : 0][2 + r] = l2;
                    }
                }
            }
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
                if (!dead)
                    dead = !__all_sync(0xffffffffu, !s_flag[0] && mbar_wait(&full[s], (unsigned)(i / NS) & 1u));
                if (dead) {
                    s_flag[0] = 1;
                    continue;
                }
                const int kb = sp.block(first + e) * kPdKeys + 16 * wl;  // this warp's 16 keys
                if (kb < sp.len && (kb + 16 > sp.lo || kb < sp.sk)) {
                    const unsigned char *st = sm + s * kPdStage;
                    float s0[4] = {0.f, 0.f, 0.f, 0.f}, s1[4] = {0.f, 0.f, 0.f, 0.f};
                    {
                        const int row = 16 * wl + (lane & 7) + ((lane >> 4) << 3);
                        const int half = (lane >> 3) & 1;
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            uint32_t b0_, b1_, b2_, b3_;
                            ldsm_x4(st + (ks >> 2) * kPdBox + am_swz(row, 2 * (ks & 3) + half), b0_, b1_, b2_, b3_);
                            mma_bf16_16816(s0, qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b0_, b1_);
                            mma_bf16_16816(s1, qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b2_, b3_);
                            if (RPT == 2) {
                                const int kq = RPT == 2 ? ks : 0;
                                mma_bf16_16816(s0, ql[kq][0], ql[kq][1], ql[kq][2], ql[kq][3], b0_, b1_);
                                mma_bf16_16816(s1, ql[kq][0], ql[kq][1], ql[kq][2], ql[kq][3], b2_, b3_);
                            }
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
                        // one of the 16 keys is visible, so mx is a logit.  Raise the
                        // running maximum only past the margin: until then p <= 2^kAmLazy.
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
                        const float p0 = exp2f(x0 - m[r]), p1 = exp2f(x1 - m[r]), p2 = exp2f(x2 - m[r]),
                                    p3 = exp2f(x3 - m[r]);
                        l[r] += (p0 + p1) + (p2 + p3);
                        ph[r][0] = pack_bf16x2(p0, p1);
                        ph[r][1] = pack_bf16x2(p2, p3);
                        pl[r][0] = pack_bf16x2(p0 - bf16lo(ph[r][0]), p1 - bf16hi(ph[r][0]));
                        pl[r][1] = pack_bf16x2(p2 - bf16lo(ph[r][1]), p3 - bf16hi(ph[r][1]));
                    }
                    {
                        const int row = 16 * wl + (lane & 7) + (((lane >> 3) & 1) << 3);
                        const int half = lane >> 4;
#pragma unroll
                        for (int n2 = 0; n2 < 8; ++n2) {
                            uint32_t w0, w1, w2, w3;
                            ldsm_x4_t(st + (2 + (n2 >> 2)) * kPdBox + am_swz(row, 2 * (n2 & 3) + half), w0, w1, w2, w3);
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
            if (RPT == 1) {  // rows gid + 8 held the P_lo . V half of the same head
#pragma unroll
                for (int t = 0; t < 16; ++t) {
                    o[t][0] += o[t][2];
                    o[t][1] += o[t][3];
                }
            }
#pragma unroll
            for (int r = 0; r < RPT; ++r) {
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
                l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
            }
            // ---- group 1 hands its state to group 0 (warp wl to warp wl, same
            //      lanes), whose warps then lay theirs out for the merge ----
            auto put = [&]() {
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    const int hd = gid + 8 * r;
                    if (hd < a.g) {
#pragma unroll
                        for (int t = 0; t < 16; ++t)
                            *reinterpret_cast<float2 *>(&s_o[(wl * GM + hd) * D + 8 * t + 2 * c]) =
                                make_float2(o[t][2 * r], o[t][2 * r + 1]);
                        if (c == 0) {
                            s_ml[(wl * GM + hd) * 2 + 0] = m[r];
                            s_ml[(wl * GM + hd) * 2 + 1] = l[r];
                        }
                    }
                }
            };
            if (grp == 1) put();
            asm volatile("bar.sync 1, %0;" ::"n"(kAmWarps * 32) : "memory");
            if (grp == 0) {
#pragma unroll
                for (int r = 0; r < RPT; ++r) {
                    const int hd = gid + 8 * r;
                    if (hd < a.g) {
                        const float m1 = s_ml[(wl * GM + hd) * 2 + 0], l1 = s_ml[(wl * GM + hd) * 2 + 1];
                        const float M = fmaxf(m[r], m1);
                        const float w0 = m[r] == -INFINITY ? 0.f : exp2f(m[r] - M);
                        const float w1 = m1 == -INFINITY ? 0.f : exp2f(m1 - M);
#pragma unroll
                        for (int t = 0; t < 16; ++t) {
                            const float2 x = *reinterpret_cast<const float2 *>(&s_o[(wl * GM + hd) * D + 8 * t + 2 * c]);
                            o[t][2 * r] = o[t][2 * r] * w0 + x.x * w1;
                            o[t][2 * r + 1] = o[t][2 * r + 1] * w0 + x.y * w1;
                        }
                        l[r] = l[r] * w0 + l1 * w1;
                        m[r] = M;
                    }
                }
                __syncwarp();  // a warp reads and writes only its own part
                put();
                asm volatile("bar.sync 2, %0;" ::"n"(kAmGroupWarps * 32) : "memory");

                // ---- group 0 merges its warps; thread = dimension ----
                const bool whole = pair_start >= u0 && pair_end <= u1;
                const int cf = whole ? cta : am_cta_of(U, G, pair_start);
                auto emit = [&](int hrow, float num, float M, float den) {
                    const int64_t row = (int64_t)b * a.nq + j * a.g + hrow;
                    if (a.own_o) {
                        a.own_o[row * D + tid] = num;
                        if (tid == 0) {
                            a.own_ml[row * 2] = M;
                            a.own_ml[row * 2 + 1] = den;
                        }
                    } else {
                        store_act(a.o, a.o_f32, row * D + tid, num / den);
                        if (a.lse && tid == 0) a.lse[row] = (M + log2f(den)) * 0.6931471805599453f;
                    }
                };
                const int slot = 2 * cta + (pair_start > u0 ? 1 : 0);
                for (int hrow = 0; hrow < a.g; ++hrow) {
                    float M = -INFINITY;
#pragma unroll
                    for (int w = 0; w < kAmGroupWarps; ++w) M = fmaxf(M, s_ml[(w * GM + hrow) * 2]);
                    float num = 0.f, den = 0.f;
#pragma unroll
                    for (int w = 0; w < kAmGroupWarps; ++w) {
                        const float mi = s_ml[(w * GM + hrow) * 2];
                        const float wt = mi == -INFINITY ? 0.f : exp2f(mi - M);
                        num += wt * s_o[(w * GM + hrow) * D + tid];
                        den += wt * s_ml[(w * GM + hrow) * 2 + 1];
                    }
                    if (whole) {
                        emit(hrow, num, M, den);
                    } else {
                        a.part_o[((int64_t)slot * a.g + hrow) * D + tid] = num;
                        if (tid == 0) {
                            a.part_ml[((int64_t)slot * a.g + hrow) * 2 + 0] = M;
                            a.part_ml[((int64_t)slot * a.g + hrow) * 2 + 1] = den;
                        }
                    }
                }
                if (!whole) {
                    const int n_p = am_cta_of(U, G, pair_end - 1) - cf + 1;
                    __threadfence();
                    asm volatile("bar.sync 2, %0;" ::"n"(kAmGroupWarps * 32) : "memory");
                    if (tid == 0) {
                        const unsigned prev = atomicAdd(&a.tickets[cf], 1u);
                        s_flag[1] = prev == (unsigned)(n_p - 1);
                        if (prev >= (unsigned)n_p) record_error(2u);
                    }
                    asm volatile("bar.sync 2, %0;" ::"n"(kAmGroupWarps * 32) : "memory");
                    if (s_flag[1]) {
                        // ---- the last CTA of the pair: partials in CTA order ----
                        __threadfence();
                        float *s_mlp = s_o;                          // [n_p][g][2]
                        float *s_w = s_o + 2 * GM * kPagedMaxCtas;   // [n_p][GM]
                        float *s_M = s_misc, *s_den = s_misc + GM;
                        // CTA cf's part of the pair is its second segment when its range begins before the pair
                        const int slot0 = 2 * cf + (am_start(U, G, cf) < pair_start ? 1 : 0);
                        auto slot_of = [&](int x) { return x == 0 ? slot0 : 2 * (cf + x); };
                        for (int x = tid; x < n_p * a.g; x += kAmGroupWarps * 32) {
                            const float2 ml = __ldcg(reinterpret_cast<const float2 *>(a.part_ml) +
                                                     (int64_t)slot_of(x / a.g) * a.g + x % a.g);
                            s_mlp[2 * x] = ml.x;
                            s_mlp[2 * x + 1] = ml.y;
                        }
                        asm volatile("bar.sync 2, %0;" ::"n"(kAmGroupWarps * 32) : "memory");
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
                        asm volatile("bar.sync 2, %0;" ::"n"(kAmGroupWarps * 32) : "memory");
                        for (int hrow = 0; hrow < a.g; ++hrow) {
                            float num = 0.f;
#pragma unroll 8
                            for (int x = 0; x < n_p; ++x)
                                num += s_w[x * GM + hrow] *
                                       __ldcg(a.part_o + ((int64_t)slot_of(x) * a.g + hrow) * D + tid);
                            emit(hrow, num, s_M[hrow], s_den[hrow]);
                        }
                        if (tid == 0) atomicExch(&a.tickets[cf], 0u);
                    }
                }
            }
            // the merge area is rewritten by the next segment
            asm volatile("bar.sync 1, %0;" ::"n"(kAmWarps * 32) : "memory");
            pair_start = pair_end;
            if (i < n && ++j == v.nkv) {
                j = 0;
                do ++b;
                while (s_start[b + 1] == s_start[b]);
                sp = pd_span(a, paged_len(v, b));
            }
        }
    }
    __syncthreads();
    if (s_flag[0] && threadIdx.x == 0) {
        record_error(8u);
        // wait (bounded) for the copies still in flight before the CTA exits
        const int issued = s_flag[2];
        for (int x = issued - NS > 0 ? issued - NS : 0; x < issued; ++x)
            mbar_wait(&full[x % NS], (unsigned)(x / NS) & 1u);
    }
}

}  // namespace tpl
