// Attention of a chunk of new tokens over a cache, bf16, both products on the
// tcgen05 tensor cores, work split over the context (chunk_plan.cuh).
//
// Row r = j G + (h mod G) of a row tile is query head h of new token j, so all
// query heads of a KV head share each K/V tile that is loaded.  Per key tile
// (128 positions) and half x of the CTA (x = 0, 1):
//   S_x = Q_x K^T     fp32 in tensor memory;
//   P_x = 2^(S_x - m) one thread per row, in bf16 against a reference maximum m
//                     that moves only when the row maximum exceeds it by more
//                     than 8 (O_x and the row sum are then rescaled), its sum
//                     taken over the bf16 values that the product uses;
//   O_x += P_x V      P from tensor memory, V MN-major from its TMA tile.
//
// Two shapes of a row tile, chosen by the rows that the longest chunk has:
//   C = 0 (more than 128 rows): 256 rows, 128 in each half, every half over all
//          128 keys of a tile.  Bound by the tensor cores and the exponentials.
//   C = 1, 2, 4 (at most 128 / C rows): bound by the cache's bytes.  The matrix
//          instruction has 128 rows whatever is in them, so the rows are put
//          there 2 C times, C copies in each half: half x takes keys 64 x .. +63
//          of every tile (N = 64 scores, K = 64 values: no product is done
//          twice), and copy i of it forms the exponentials of 64 / C of those
//          keys only; the other columns of its P stay zero.  The copies' results
//          are merged at the end of a segment.  With one copy of 32 rows a
//          single warp would form 4096 exponentials per tile, longer than the
//          tile's bytes take; with 8 copies each warp forms 512.
//
// Masked tiles.  A weight of 0 times a value that is not finite is not 0, so in
// a tile that some row does not see whole, the value rows outside the row
// tile's span are zeroed in shared memory, and where another value is not
// finite it is zeroed too and added, by hand, to the rows that see its key.
//
// Warps: 0 = K loader, 10 = V loader, 1 = MMA issuer and tensor-memory owner,
// 2..5 = half 0, 6..9 = half 1 (they also load the queries).
// Rings and barriers run on across the segments of a CTA: the producer is
// already loading the next segment's tiles, and the next queries are in place,
// while a segment's result is written.  Every wait is bounded; on a timeout
// the kernel records YOCOPP_ETIMEOUT, waits (bounded) for what it has in
// flight, frees the tensor memory and returns.
#pragma once

#include "chunk_plan.cuh"
#include "prefill_attn_tc.cuh"

namespace yocopp {

template <int D, int C>
struct ChunkTc {
    static constexpr bool PAIR = C == 0;
    static constexpr int RT = PAIR ? 256 : 128 / (PAIR ? 1 : C);  // rows of a row tile
    static constexpr int TK = 128;                                 // positions of a key tile
    static constexpr int XK = PAIR ? 128 : 64;                     // keys of a half's products
    static constexpr int NK = PAIR ? 128 : 64 / (PAIR ? 1 : C);    // keys whose exponentials a thread forms
    static constexpr int NBOX = D / 64, BOXB = 128 * 128, TILE_BYTES = NBOX * BOXB;
    static constexpr int SCR_BYTES = PAIR ? 0 : 256 * 128;         // merge of the copies: 256 x 32 fp32
    static constexpr int KSLOTS = D == 64 ? 4 : (PAIR ? 2 : 3), VSLOTS = D == 64 ? 4 : 2;
    static constexpr int Q_OFF = 0;
    static constexpr int SCR_OFF = (PAIR ? 2 : 1) * TILE_BYTES;
    static constexpr int K_OFF = SCR_OFF + SCR_BYTES;
    static constexpr int V_OFF = K_OFF + KSLOTS * TILE_BYTES;
    static constexpr int BAR_OFF = V_OFF + VSLOTS * TILE_BYTES;
    // q_full[2], k_full, k_empty, v_full, v_empty, s_full[2], p_full[2], o_last[2], drain
    static constexpr int NBAR = 2 + 2 * KSLOTS + 2 * VSLOTS + 7;
    static constexpr int SMEM = 1024 + BAR_OFF + NBAR * 8;
    static constexpr int THREADS = 352;
    static constexpr uint32_t IDESC_QK = umma_idesc_bf16(128, XK, false);
    static constexpr uint32_t IDESC_PV = umma_idesc_bf16(128, D, true);
    // tensor memory: S_x at 128 x (PAIR: P_x over its first 64 columns; else P_x at 128 x + 64), O_x at 256 + 128 x
    static constexpr int TMEM_COLS = 512, P_COL = PAIR ? 0 : 64;
    static constexpr float RESCALE_SLACK = 8.f;
};
static_assert(ChunkTc<128, 0>::SMEM <= 232448 - 512 && ChunkTc<128, 1>::SMEM <= 232448 - 512 &&
                  ChunkTc<64, 0>::SMEM <= 232448 - 512 && ChunkTc<64, 1>::SMEM <= 232448 - 512,
              "chunk shared memory");

// max of three that keeps a NaN
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ bool bf16x2_not_finite(uint32_t w) {
    return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}

// Bits of the positions base .. base + 31 that a row sees.
__device__ __forceinline__ uint32_t sight_bits(const ChunkSight& s, int base) {
    if (!s.tree) {
        const int a = max(s.lo - base, 0), b = min(s.hi - base, 31);  // bits a..b
        if (a > b) return 0u;
        return (0xFFFFFFFFu << a) & (0xFFFFFFFFu >> (31 - b));
    }
    const int c = base - s.p0;  // chunk position of bit 0
    if (c >= 64) return 0u;
    if (c <= -32) return 0xFFFFFFFFu;
    if (c >= 0) return uint32_t(s.bits >> c);
    return ((1u << -c) - 1u) | (uint32_t(s.bits) << -c);
}

template <int D, int C>
__global__ void __launch_bounds__(ChunkTc<D, C>::THREADS, 1)
chunk_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ ChunkParams p) {
    using S = ChunkTc<D, C>;
    constexpr bool PAIR = S::PAIR;
    constexpr int TK = S::TK, RT = S::RT, NK = S::NK;
    extern __shared__ uint8_t smem_raw[];
    __shared__ volatile int s_abort;
    __shared__ int s_cdone;
    __shared__ uint32_t s_tmem;
    __shared__ unsigned s_bad[4];          // keys of a masked tile with a value that is not finite
    __shared__ int64_t s_scan[S::THREADS / 32];
    __shared__ ChunkStart s_start;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cta = blockIdx.x;
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* q_full = reinterpret_cast<uint64_t*>(base + S::BAR_OFF);  // [2]
    uint64_t* k_full = q_full + 2;
    uint64_t* k_empty = k_full + S::KSLOTS;
    uint64_t* v_full = k_empty + S::KSLOTS;
    uint64_t* v_empty = v_full + S::VSLOTS;
    uint64_t* s_full = v_empty + S::VSLOTS;  // [2]
    uint64_t* p_full = s_full + 2;           // [2]
    uint64_t* o_last = p_full + 2;           // [2]
    uint64_t* drain = o_last + 2;

    if (tid == 0) {
        for (int s = 0; s < S::KSLOTS; ++s) {
            mbar_init(&k_full[s], 1);
            mbar_init(&k_empty[s], 1);
        }
        for (int s = 0; s < S::VSLOTS; ++s) {
            mbar_init(&v_full[s], 1);
            mbar_init(&v_empty[s], 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&q_full[x], 4);
            mbar_init(&s_full[x], 1);
            mbar_init(&p_full[x], 4);
            mbar_init(&o_last[x], 1);
        }
        mbar_init(drain, 1);
        fence_mbar_init();
        s_abort = 0;
        s_cdone = 0;
        s_bad[0] = s_bad[1] = s_bad[2] = s_bad[3] = 0u;
    }
    // before the wait: nothing here depends on the previous kernel
    if (warp == 0 && lane == 0) prefetch_tensormap(&tmK);
    if (warp == 10 && lane == 0) prefetch_tensormap(&tmV);
    if (warp == 1) {
        tmem_alloc(&s_tmem, S::TMEM_COLS);
        tmem_relinquish();
    }
    griddep_launch_dependents();  // the merge's blocks take their places beside these CTAs and wait for their end
    griddep_wait();
    tc_fence_before();
    chunk_find_start<RT, TK>(p, cta, s_scan, &s_start);  // ends with a block-wide barrier
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    if (s_start.item >= s_start.end) {  // nothing for this CTA
        if (tid == 0) __stcg(&p.desc[cta].last_cta, -1);
        if (warp == 1) tmem_dealloc(tmem, S::TMEM_COLS);
        return;
    }
    ChunkWalk<RT, TK> walk(p, s_start);
    ChunkSegment sg;
    // does half 1 have rows in this segment
    auto both = [&](const ChunkSegment& g) { return !PAIR || g.s.n * p.G > g.rt * RT + 128; };

    if (warp == 0 || warp == 10) {
        // ------------------------------------------------------------------ loaders
        const bool kl = warp == 0;
        const CUtensorMap* map = kl ? &tmK : &tmV;
        uint64_t* full = kl ? k_full : v_full;
        uint64_t* empty = kl ? k_empty : v_empty;
        uint8_t* ring = base + (kl ? S::K_OFF : S::V_OFF);
        const int slots = kl ? S::KSLOTS : S::VSLOTS;
        int slot = 0, round = 0, issued = 0;
        bool ok = true;
        while (ok && walk.next(sg)) {
            for (int t = sg.t0; t < sg.t1; ++t) {
                // the table is read before the wait for the slot
                const int crow = chunk_box_row<TK>(p, sg, t, lane);
                const unsigned boxes = __ballot_sync(0xffffffffu, crow >= 0);
                if (lane == 0) ok = !s_abort && mbar_wait(&empty[slot], (round & 1) ^ 1, p.wait_limit_ns);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
                if (!(kl && cta == 0 && sg.item + (t - sg.t0) == p.drop_tile)) {  // failure injection (tests)
                    if (lane == 0)
                        mbar_arrive_expect_tx(&full[slot], uint32_t(__popc(boxes) * p.boxr * 128 * S::NBOX));
                    __syncwarp();
                    if (crow >= 0) {
#pragma unroll
                        for (int bx = 0; bx < S::NBOX; ++bx)
                            tma_load_2d(ring + slot * S::TILE_BYTES + bx * S::BOXB + lane * p.boxr * 128, map,
                                        &full[slot], bx * 64, crow);
                    }
                }
                ++issued;
                if (++slot == slots) {
                    slot = 0;
                    ++round;
                }
            }
        }
        if (!ok) {
            record_status(YOCOPP_ETIMEOUT);
            s_abort = 1;
        }
        if (!ok || s_abort)  // the copies in flight land before the CTA can exit
            for (int t = max(0, issued - slots); t < issued; ++t)
                (void)mbar_wait(&full[t % slots], (t / slots) & 1, p.wait_limit_ns);
        return;
    }

    if (warp == 1) {
        // ------------------------------------------------------------- MMA issuer
        if (lane == 0) {
            const uint32_t qaddr = smem_addr(base + S::Q_OFF);
            const uint32_t kaddr = smem_addr(base + S::K_OFF);
            const uint32_t vaddr = smem_addr(base + S::V_OFF);
            int ks = 0, kr = 0, vs = 0, vr = 0;  // next tile's slot and round of the rings
            int np[2] = {0, 0};                  // tiles so far of each half
            int nq[2] = {0, 0};                  // segments so far of each half
            bool ok = true, issued_any = false;
            auto qk = [&](int x) {
                const uint32_t ka = kaddr + uint32_t(ks * S::TILE_BYTES + (PAIR ? 0 : x * 64 * 128));
                const uint32_t qa = qaddr + uint32_t(PAIR ? x * S::TILE_BYTES : 0);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = uint32_t((kk >> 2) * S::BOXB + (kk & 3) * 32);
                    umma_bf16(tmem + 128 * x, umma_desc_sw128(qa + off), umma_desc_sw128(ka + off), S::IDESC_QK,
                              kk > 0 ? 1u : 0u);
                }
                umma_commit(&s_full[x]);
                issued_any = true;
            };
            auto pv = [&](int x, bool last) {
                const uint32_t va = vaddr + uint32_t(vs * S::TILE_BYTES + (PAIR ? 0 : x * 64 * 128));
#pragma unroll
                for (int kk = 0; kk < S::XK / 16; ++kk)  // O starts from zeros that the softmax threads wrote
                    umma_bf16_tmem_a(tmem + 256 + 128 * x, tmem + 128 * x + S::P_COL + 8 * kk,
                                     umma_desc_sw128_mn(va + uint32_t(kk * 16 * 128), S::BOXB, 1024), S::IDESC_PV, 1u);
                if (last) umma_commit(&o_last[x]);
                issued_any = true;
            };
            auto next_k = [&]() {
                if (++ks == S::KSLOTS) {
                    ks = 0;
                    ++kr;
                }
            };
            while (ok && walk.next(sg)) {
                const bool two = both(sg);
                const int nt = sg.t1 - sg.t0;
                ok = !s_abort && (!PAIR || mbar_wait(&q_full[0], nq[0] & 1, p.wait_limit_ns)) &&
                     (!two || mbar_wait(&q_full[1], nq[1] & 1, p.wait_limit_ns)) &&
                     mbar_wait(&k_full[ks], kr & 1, p.wait_limit_ns);
                if (!ok) break;
                ++nq[0];
                if (two) ++nq[1];
                tc_fence_after();
                qk(0);
                if (two) qk(1);
                umma_commit(&k_empty[ks]);
                next_k();
                for (int i = 0; i < nt; ++i) {
                    const bool more = i + 1 < nt;
                    // half 0: P V of tile i, then S of tile i + 1; the same for half 1
                    ok = !s_abort && mbar_wait(&p_full[0], np[0]++ & 1, p.wait_limit_ns) &&
                         mbar_wait(&v_full[vs], vr & 1, p.wait_limit_ns);
                    if (!ok) break;
                    tc_fence_after();
                    pv(0, !more);
                    if (more) {
                        ok = mbar_wait(&k_full[ks], kr & 1, p.wait_limit_ns);
                        if (!ok) break;
                        tc_fence_after();
                        qk(0);
                    }
                    if (two) {
                        ok = !s_abort && mbar_wait(&p_full[1], np[1]++ & 1, p.wait_limit_ns);
                        if (!ok) break;
                        tc_fence_after();
                        pv(1, !more);
                        if (more) qk(1);
                    }
                    umma_commit(&v_empty[vs]);
                    if (++vs == S::VSLOTS) {
                        vs = 0;
                        ++vr;
                    }
                    if (more) {
                        umma_commit(&k_empty[ks]);
                        next_k();
                    }
                }
            }
            if (!ok) {
                record_status(YOCOPP_ETIMEOUT);
                s_abort = 1;
            }
            if (issued_any) {  // every product issued finishes before the tensor memory is freed
                umma_commit(drain);
                (void)mbar_wait(drain, 0, p.wait_limit_ns);
            }
            // the softmax warps finish reading O before the tensor memory is freed
            const uint64_t t0 = globaltimer_ns();
            while (atomicAdd(&s_cdone, 0) < 8 && globaltimer_ns() - t0 <= p.wait_limit_ns) __nanosleep(64);
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, S::TMEM_COLS);
        return;
    }

    // ------------------------------------------------------------ softmax + epilogue
    const int x = (warp - 2) >> 2;                  // half
    const int qd = warp & 3;
    const int r = 32 * qd + lane;                   // row of the half (tensor-memory lane)
    const int copy = PAIR ? 0 : r / RT;             // PAIR: unused
    const int row = PAIR ? 128 * x + r : r % RT;    // row of the row tile
    const int kofs = PAIR ? 0 : 64 * x + NK * copy; // first key of the tile that this thread takes
    const uint32_t lanes = uint32_t(32 * qd) << 16;
    const uint32_t tS = tmem + 128 * x + lanes;
    const uint32_t tP = tS + S::P_COL;
    const uint32_t tO = tmem + 256 + 128 * x + lanes;
    uint8_t* scr = base + S::SCR_OFF;

    // the queries of a segment's row tile into their swizzled tile (split: half 1 loads the one tile,
    // whose last product is the last that half 1 has seen done)
    auto load_q = [&](const ChunkSegment& g) {
        if (!PAIR && x == 0) return;
        constexpr int CH = D / 8, RPI = 32 / CH, IT = 32 / RPI;  // chunks of a row, rows per pass, passes
        const int ch = lane % CH;
        const int rows_all = g.s.n * p.G;
        uint4 v[IT];
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int rr = 32 * qd + i * RPI + lane / CH;
            const int R = g.rt * RT + (PAIR ? 128 * x + rr : rr % RT);
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (R < rows_all) {
                const int j = chunk_token(p, R);
                v[i] = ld_stream(p.q + ((int64_t(g.s.row0) + j) * p.hq + g.g * p.G + (R - j * p.G)) * (D * 2) + ch * 16);
            }
        }
        uint8_t* q = base + S::Q_OFF + (PAIR ? x * S::TILE_BYTES : 0);
#pragma unroll
        for (int i = 0; i < IT; ++i) {
            const int rr = 32 * qd + i * RPI + lane / CH;
            *reinterpret_cast<uint4*>(q + (ch >> 3) * S::BOXB + rr * 128 + (((ch & 7) ^ (rr & 7)) << 4)) = v[i];
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[x]);
    };
    // The softmax warps' own barriers are named ones: all of them come to every one, whatever happens, as a
    // wait that has run out (ok = false) changes no branch around a barrier; it only makes later waits be
    // skipped.  Barrier 1: both halves, 2: half 0 alone.
    auto meet = [&](bool two) {
        if (two) asm volatile("bar.sync 1, 256;" ::: "memory");
        else asm volatile("bar.sync 2, 128;" ::: "memory");
    };
    bool ok = true;
    auto await = [&](uint64_t* bar, int parity) {
        if (ok) ok = !s_abort && mbar_wait(bar, parity, p.wait_limit_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) s_abort = 1;
    };

    if constexpr (!PAIR) {  // the columns of P that belong to other copies stay zero
        uint32_t z[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = 0u;
        tmem_st32u(tP, z);
    }
    bool split_end = false;                          // this CTA leaves its last row tile unfinished
    int n_x = 0, n_seg = 0, vs = 0, vr = 0;
    bool have = walk.next(sg);
    if (have && (x == 0 || both(sg))) load_q(sg);
    while (have) {
        const ChunkSegment g = sg;
        const bool two = both(g);
        const int nt = g.t1 - g.t0;
        const bool mine = x == 0 || two;
        if (g.t0 == g.u0 && g.t1 < g.u1) {
            split_end = true;
            if (warp == 2 && lane == 0) {
                ChunkDesc* d = p.desc + cta;
                __stcg(&d->row0, g.s.row0);
                __stcg(&d->first_row, g.rt * RT);
                __stcg(&d->rows, min(RT, g.s.n * p.G - g.rt * RT));
                __stcg(&d->g, g.g);
                __stcg(&d->last_cta, chunk_cta_of(s_start.total, g.item + (g.u1 - g.u0) - 1, p.num_ctas));
            }
        }
        float m_ref = NEG_INF_F, l = 0.f;
        const int R = g.rt * RT + row;               // row of the sequence
        const int rows_all = g.s.n * p.G;
        if (mine) {
            const int j = min(chunk_token(p, R), g.s.n - 1);
            ChunkSight see = chunk_sight(p, g.s, j);
            if (see.tree && g.s.n < 64) see.bits &= (1ull << g.s.n) - 1ull;
            // positions that every row of the row tile sees: [lo_all, hi_all]
            const int j0 = chunk_token(p, g.rt * RT);
            const int j1 = min(chunk_token(p, g.rt * RT + RT - 1), g.s.n - 1);
            const int hi_all = p.tree ? g.s.p0 - 1 : g.s.p0 + j0;
            const int lo_all = !p.tree && p.window ? max(0, g.s.p0 + j1 + 1 - p.window) : 0;
            {
                float z[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = 0.f;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) tmem_st32(tO + uint32_t(c * 32), z);
            }
            for (int t = g.t0; t < g.t1; ++t) {
                await(&s_full[x], n_x & 1);
                ++n_x;
                tc_fence_after();
                const int key0 = t * TK;
                const bool masked = key0 + TK - 1 > hi_all || key0 < lo_all;
                uint32_t u[NK];
                if constexpr (NK == 16) {
                    tmem_ld16_nowait(tS + uint32_t(NK * copy), u);
                } else {
#pragma unroll
                    for (int c = 0; c < NK / 32; ++c)
                        tmem_ld32_nowait(tS + uint32_t((PAIR ? 0 : NK * copy) + c * 32),
                                         *reinterpret_cast<uint32_t(*)[32]>(&u[c * 32]));
                }
                tmem_wait_ld();
                if (masked) {
#pragma unroll
                    for (int w = 0; w < (NK + 31) / 32; ++w) {
                        const uint32_t bits = sight_bits(see, key0 + kofs + 32 * w);
#pragma unroll
                        for (int c = 0; c < (NK < 32 ? NK : 32); ++c)
                            if (!((bits >> c) & 1u)) u[32 * w + c] = __float_as_uint(NEG_INF_F);
                    }
                }
                float mx4[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) mx4[i] = __uint_as_float(u[i]);
#pragma unroll
                for (int c = 4; c < NK; c += 2)
                    mx4[(c >> 1) & 3] = fmax3_nan(mx4[(c >> 1) & 3], __uint_as_float(u[c]), __uint_as_float(u[c + 1]));
                const float mx = fmax3_nan(fmax3_nan(mx4[0], mx4[1], mx4[2]), mx4[3], mx4[3]);
                const float m_new = fmaxf(m_ref, mx * p.qscale);
                const bool rescale = m_new > m_ref + S::RESCALE_SLACK;
                const float corr = rescale ? ex2_approx(m_ref - m_new) : 1.f;
                if (rescale) {
                    l *= corr;
                    m_ref = m_new;
                }
                if (!(mx < -NEG_INF_F)) {  // a score of +inf or NaN makes the row NaN
                    l = mx - mx;
                    if (m_ref == NEG_INF_F) m_ref = 0.f;
                }
                const float nmsub = m_ref == NEG_INF_F ? 0.f : -m_ref;
                const float2 qs2 = make_float2(p.qscale, p.qscale), nm2 = make_float2(nmsub, nmsub);
                float2 ls[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                constexpr int W = NK >= 64 ? 32 : NK / 2;  // packed pairs of one store
#pragma unroll
                for (int c = 0; c < NK / 2 / W; ++c) {
                    uint32_t pw[W];
#pragma unroll
                    for (int e = 0; e < W; ++e) {
                        const int k = 2 * (W * c + e);
                        const float2 xv = ffma2(make_float2(__uint_as_float(u[k]), __uint_as_float(u[k + 1])), qs2, nm2);
                        // a quarter of the exponentials on the FMA pipe where the tensor cores are the bound
                        const float2 pe = PAIR && poly_pair(e) ? exp2_poly2(xv)
                                                               : make_float2(ex2_approx(xv.x), ex2_approx(xv.y));
                        pw[e] = float2_to_bf16x2(pe.x, pe.y);
                        ls[e & 1] = add_bf16x2(ls[e & 1], pw[e]);
                    }
                    const uint32_t at = tP + uint32_t((PAIR ? 0 : NK / 2 * copy) + c * W);
                    if constexpr (W == 32) tmem_st32u(at, pw);
                    else if constexpr (W == 16) tmem_st16u(at, pw);
                    else tmem_st8u(at, pw);
                }
                l += (ls[0].x + ls[1].x) + (ls[0].y + ls[1].y);
                if (t > g.t0 && __any_sync(0xffffffffu, rescale)) {
                    // S of this tile was issued after P V of the previous one, so O is complete up to there
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        float o[32];
                        tmem_ld32(tO + uint32_t(c * 32), o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= corr;
                        tmem_st32(tO + uint32_t(c * 32), o);
                    }
                }
                if (masked) {
                    // key row r of the value tile, this half's part of its chunks
                    await(&v_full[vs], vr & 1);
                    constexpr int CH = D / 8;
                    const int c0 = two && x == 1 ? CH / 2 : 0, c1 = two && x == 0 ? CH / 2 : CH;
                    uint8_t* vrow = base + S::V_OFF + vs * S::TILE_BYTES + r * 128;
                    const bool outside = key0 + r < g.span.lo || key0 + r > g.span.hi;
                    bool bad = false;
                    for (int ch = c0; ch < c1; ++ch) {
                        uint4* a = reinterpret_cast<uint4*>(vrow + (ch >> 3) * S::BOXB + (((ch & 7) ^ (r & 7)) << 4));
                        if (outside) {
                            *a = make_uint4(0u, 0u, 0u, 0u);
                        } else {
                            const uint4 w = *a;
                            bad |= bf16x2_not_finite(w.x) | bf16x2_not_finite(w.y) | bf16x2_not_finite(w.z) |
                                   bf16x2_not_finite(w.w);
                        }
                    }
                    if (bad) atomicOr(&s_bad[r >> 5], 1u << (r & 31));
                    meet(two);
                    const volatile unsigned* vb = s_bad;
                    const unsigned any = vb[0] | vb[1] | vb[2] | vb[3];
                    if (any) {  // uniform over the CTA's softmax threads
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            float o[32];
                            tmem_ld32(tO + uint32_t(c * 32), o);
                            for (int k = kofs; k < kofs + NK; ++k) {
                                if (!((vb[k >> 5] >> (k & 31)) & 1u) || !see.sees(key0 + k)) continue;
                                const uint8_t* kr = base + S::V_OFF + vs * S::TILE_BYTES + k * 128 + (c >> 1) * S::BOXB;
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    const int ch = (c & 1) * 4 + i / 8;
                                    const uint32_t h = *reinterpret_cast<const uint16_t*>(
                                        kr + ((ch ^ (k & 7)) << 4) + (i & 7) * 2);
                                    if ((h & 0x7F80u) == 0x7F80u) o[i] += __uint_as_float(h << 16);
                                }
                            }
                            __syncwarp();
                            tmem_st32(tO + uint32_t(c * 32), o);
                        }
                        meet(two);
                        if (bad) {
                            for (int ch = c0; ch < c1; ++ch) {
                                uint16_t* a = reinterpret_cast<uint16_t*>(vrow + (ch >> 3) * S::BOXB +
                                                                          (((ch & 7) ^ (r & 7)) << 4));
                                for (int i = 0; i < 8; ++i)
                                    if ((a[i] & 0x7F80u) == 0x7F80u) a[i] = 0;
                            }
                        }
                        if (x == 0 && r < 4) s_bad[r] = 0u;
                    }
                    fence_proxy_async_smem();
                }
                if (++vs == S::VSLOTS) {
                    vs = 0;
                    ++vr;
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[x]);
            }
        } else {
            for (int t = 0; t < nt; ++t)
                if (++vs == S::VSLOTS) {
                    vs = 0;
                    ++vr;
                }
        }
        have = walk.next(sg);
        if (have && (x == 0 || both(sg))) load_q(sg);
        if (!mine) continue;

        // ---- the segment's result: whole row tiles to the output, others to the workspace
        await(&o_last[x], n_seg & 1);
        ++n_seg;
        tc_fence_after();
        const bool whole = g.t0 == g.u0 && g.t1 == g.u1;
        float* slot = chunk_slot<RT, D>(p, cta, g.t0 == g.u0 ? 1 : 0);
        if constexpr (PAIR) {
            const bool store = R < rows_all;
            const bool none = m_ref == NEG_INF_F;
            const float w = !whole ? 1.f : none ? 0.f : 1.f / l;
            const int j = chunk_token(p, R);
            uint8_t* orow = p.out + ((int64_t(g.s.row0) + j) * p.hq + g.g * p.G + (R - j * p.G)) * int64_t(D * 2);
            if (!whole && store) {
                __stcg(slot + RT * D + row, m_ref);
                __stcg(slot + RT * D + RT + row, l);
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
                tmem_ld32(tO + uint32_t(c * 32), o);
                if (!store) continue;
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = none ? 0.f : o[i] * w;
#pragma unroll
                    for (int q4 = 0; q4 < 4; ++q4)
                        st_global(orow + (c * 32 + q4 * 8) * 2,
                                  make_uint4(float2_to_bf16x2(o[q4 * 8 + 0], o[q4 * 8 + 1]),
                                             float2_to_bf16x2(o[q4 * 8 + 2], o[q4 * 8 + 3]),
                                             float2_to_bf16x2(o[q4 * 8 + 4], o[q4 * 8 + 5]),
                                             float2_to_bf16x2(o[q4 * 8 + 6], o[q4 * 8 + 7])));
                } else {
#pragma unroll
                    for (int q4 = 0; q4 < 8; ++q4)
                        __stcg(reinterpret_cast<float4*>(slot + int64_t(row) * D + c * 32 + q4 * 4),
                               make_float4(o[q4 * 4], o[q4 * 4 + 1], o[q4 * 4 + 2], o[q4 * 4 + 3]));
                }
            }
        } else {
            constexpr int NC = 2 * (PAIR ? 1 : C);  // copies of a row
            const int me = 128 * x + r;
            float* s_m = reinterpret_cast<float*>(scr);
            float* s_l = s_m + 256;
            s_m[me] = m_ref;
            s_l[me] = l;
            meet(true);
            float M = NEG_INF_F, L = 0.f;
#pragma unroll
            for (int i = 0; i < NC; ++i) M = fmaxf(M, s_m[RT * i + row]);
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const float mi = s_m[RT * i + row];
                L += mi == NEG_INF_F ? 0.f : s_l[RT * i + row] * ex2_approx(mi - M);
            }
            meet(true);  // read by all before it is written over
            // a row that sees nothing gives zeros
            const float w = m_ref == NEG_INF_F ? 0.f : ex2_approx(m_ref - M) * (whole ? 1.f / L : 1.f);
            if (!whole && copy == 0 && x == 0 && R < rows_all) {
                __stcg(slot + RT * D + row, M);
                __stcg(slot + RT * D + RT + row, L);
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
                tmem_ld32(tO + uint32_t(c * 32), o);
#pragma unroll
                for (int q4 = 0; q4 < 8; ++q4)
                    *reinterpret_cast<float4*>(scr + me * 128 + ((q4 ^ (me & 7)) << 4)) =
                        make_float4(o[q4 * 4] * w, o[q4 * 4 + 1] * w, o[q4 * 4 + 2] * w, o[q4 * 4 + 3] * w);
                meet(true);
#pragma unroll
                for (int i = 0; i < RT / 32; ++i) {
                    const int id = me + 256 * i, rr = id >> 3, q4 = id & 7;
                    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < NC; ++k) {
                        const int at = RT * k + rr;
                        const float4 b = *reinterpret_cast<const float4*>(scr + at * 128 + ((q4 ^ (at & 7)) << 4));
                        a.x += b.x;
                        a.y += b.y;
                        a.z += b.z;
                        a.w += b.w;
                    }
                    const int RR = g.rt * RT + rr;
                    if (RR >= rows_all) continue;
                    if (whole) {
                        const int j = chunk_token(p, RR);
                        uint2 v = make_uint2(float2_to_bf16x2(a.x, a.y), float2_to_bf16x2(a.z, a.w));
                        *reinterpret_cast<uint2*>(p.out + ((int64_t(g.s.row0) + j) * p.hq + g.g * p.G + (RR - j * p.G)) *
                                                              int64_t(D * 2) + (c * 32 + q4 * 4) * 2) = v;
                    } else {
                        __stcg(reinterpret_cast<float4*>(slot + int64_t(rr) * D + c * 32 + q4 * 4), a);
                    }
                }
                meet(true);
            }
        }
    }
    if (!ok) record_status(YOCOPP_ETIMEOUT);
    if (warp == 2 && lane == 0 && !split_end) __stcg(&p.desc[cta].last_cta, -1);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) atomicAdd(&s_cdone, 1);
}

}  // namespace yocopp
