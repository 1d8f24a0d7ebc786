// Work plan of the chunk attention, shared by its kernels and the merge.
//
// The rows of sequence b and KV head g are its new tokens' query heads of that
// group, row r = j G + (h mod G), cut into row tiles of RT rows; the keys that
// any row of a tile may see are cut into key tiles of TK positions.  Every
// (row tile, key tile) pair is one item.  The items of all sequences, in the
// order (sequence, KV head, row tile, key tile), are dealt out to the CTAs in
// equal contiguous ranges, so that one long sequence or many short ones fill
// the GPU alike.  A CTA's range is a run of segments, each a range of key
// tiles of one row tile.  A segment that is a whole row tile is written to the
// output; of the others a CTA has at most two (the end of a row tile begun by
// an earlier CTA and the start of one that a later CTA goes on with), whose
// unnormalised results go to its two slots of the workspace, and a second
// launch merges them.
#pragma once

#include "compose_append.cuh"

namespace yocopp {

struct ChunkParams {
    const uint8_t* q;            // [total_q][hq][D]
    uint8_t* out;                // [total_q][hq][D]
    const int32_t* pos;          // [batch] cache position of the first row, or null (0)
    const int32_t* cu_q;         // [batch + 1], or null (n_uniform rows each)
    const int32_t* block_table;  // null: contiguous
    const unsigned long long* tree;  // [total_q] visible chunk positions, or null (causal)
    int64_t total_q;
    int32_t n_uniform, max_q, window;
    int32_t batch, hq, hkv, G, capacity;
    uint32_t g_m, g_s;           // division by G (fast_div); rows of a sequence are below 2^31
    int32_t bs_log2, mbps, num_blocks, box_log2;
    float qscale;                // softmax scale * log2(e)
    int32_t num_ctas;            // at least 2
    uint64_t cta_m;              // ceil(2^64 / num_ctas)
    float* part;                 // [num_ctas][2][RT][D + 2]: o, then m, l
    struct ChunkDesc* desc;      // [num_ctas]
    uint64_t wait_limit_ns;
    int32_t drop_tile;           // testing: item of CTA 0 whose K load is never issued (-1: none)
};

// What the merge needs of a row tile that its CTA began and did not finish.
struct ChunkDesc {
    int32_t row0, first_row, rows, g;  // first query row of the sequence, first row of the tile, rows in it, KV head
    int32_t last_cta;                  // the CTA that ends it; -1: nothing to merge
    int32_t pad[3];
};

struct ChunkSeq {
    int row0, n, p0;
};

// Rows and first position of sequence b; n = 0 where they are not valid (recorded where `report`).
__device__ __forceinline__ ChunkSeq chunk_seq(const ChunkParams& p, int b, bool report) {
    ChunkSeq s;
    if (p.cu_q) {
        s.row0 = __ldg(p.cu_q + b);
        s.n = __ldg(p.cu_q + b + 1) - s.row0;
    } else {
        s.row0 = b * p.n_uniform;
        s.n = p.n_uniform;
    }
    s.p0 = p.pos ? __ldg(p.pos + b) : 0;
    int bad = 0;
    if (s.row0 < 0 || s.n < 0 || int64_t(s.row0) + s.n > p.total_q) bad = YOCOPP_EDEVICE_CHECK;
    else if (s.n > p.max_q || s.p0 < 0 || int64_t(s.p0) + s.n > p.capacity) bad = YOCOPP_ECAPACITY;
    if (bad) {
        if (report) record_status(bad);
        s.n = 0;
    }
    return s;
}

// New token of row r.
__device__ __forceinline__ int chunk_token(const ChunkParams& p, int r) { return int(fast_div(uint32_t(r), p.g_m, p.g_s)); }

// Positions [lo, hi] that the rows of a row tile may see.
struct ChunkSpan {
    int lo, hi;
};
template <int RT>
__device__ __forceinline__ ChunkSpan chunk_span(const ChunkParams& p, const ChunkSeq& s, int rt) {
    ChunkSpan r;
    if (p.tree) {
        r.lo = 0;
        r.hi = s.p0 + s.n - 1;
    } else {
        const int j0 = chunk_token(p, rt * RT), j1 = min(chunk_token(p, rt * RT + RT - 1), s.n - 1);
        r.lo = p.window ? max(0, s.p0 + j0 + 1 - p.window) : 0;
        r.hi = s.p0 + j1;
    }
    return r;
}
template <int RT>
__device__ __forceinline__ int chunk_row_tiles(const ChunkParams& p, const ChunkSeq& s) {
    return (s.n * p.G + RT - 1) / RT;
}
template <int RT, int TK>
__device__ __forceinline__ int64_t chunk_items_per_head(const ChunkParams& p, const ChunkSeq& s) {
    int64_t t = 0;
    const int nrt = chunk_row_tiles<RT>(p, s);
    for (int rt = 0; rt < nrt; ++rt) {
        const ChunkSpan r = chunk_span<RT>(p, s, rt);
        t += r.hi / TK - r.lo / TK + 1;
    }
    return t;
}

// One segment: key tiles [t0, t1) of row tile rt of (b, g), whose key tiles are [u0, u1).
struct ChunkSegment {
    ChunkSeq s;
    ChunkSpan span;
    int b, g, rt, t0, t1, u0, u1;
    int64_t item;  // number of its first item
};

// The CTA's place in the plan: found once by the whole CTA, then walked by every role for itself.
struct ChunkStart {
    int b, g, rt, t;
    int64_t item, end, total;
};

// first item of CTA c: total / num_ctas each, one more for the first total mod num_ctas.  The quotient by the high
// half of the product with ceil(2^64 / num_ctas), exact for total * num_ctas < 2^64; a 64-bit division is a
// subroutine of some hundred instructions.
__device__ __forceinline__ int64_t chunk_first_item(const ChunkParams& p, int64_t total, int c) {
    const int64_t q = int64_t(__umul64hi(uint64_t(total), p.cta_m)), r = total - q * p.num_ctas;
    return q * c + min(int64_t(c), r);
}
// the CTA that has an item, at or behind CTA c
__device__ __forceinline__ int chunk_cta_of(int64_t total, int c, int64_t item, const ChunkParams& p) {
    while (chunk_first_item(p, total, c + 1) <= item) ++c;
    return c;
}

// All threads of the CTA call it; `start` is shared memory.  scan: one int64 per warp, shared.
template <int RT, int TK>
__device__ __forceinline__ void chunk_find_start(const ChunkParams& p, int cta, int64_t* scan, ChunkStart* start) {
    const int tid = threadIdx.x, nthr = blockDim.x, lane = tid & 31, warp = tid >> 5, nw = nthr >> 5;
    const int per = (p.batch + nthr - 1) / nthr;
    const int b0 = min(p.batch, tid * per), b1 = min(p.batch, b0 + per);
    int64_t mine = 0;
    for (int b = b0; b < b1; ++b) mine += chunk_items_per_head<RT, TK>(p, chunk_seq(p, b, cta == 0)) * p.hkv;
    int64_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) scan[warp] = sum;
    __syncthreads();
    int64_t before = sum - mine, total = 0;
    for (int w = 0; w < nw; ++w) {
        if (w < warp) before += scan[w];
        total += scan[w];
    }
    const int64_t w0 = chunk_first_item(p, total, cta), w1 = chunk_first_item(p, total, cta + 1);
    if (w0 >= w1) {
        if (tid == 0) {
            start->item = start->end = 0;
            start->total = total;
        }
    } else if (w0 >= before && w0 < before + mine) {
        int64_t at = before;
        for (int b = b0; b < b1; ++b) {
            const ChunkSeq s = chunk_seq(p, b, false);
            const int64_t per_head = chunk_items_per_head<RT, TK>(p, s);
            if (w0 >= at + per_head * p.hkv) {
                at += per_head * p.hkv;
                continue;
            }
            int g = 0;
            int64_t rem = w0 - at;
            for (; rem >= per_head; rem -= per_head) ++g;
            int rt = 0;
            for (;; ++rt) {
                const ChunkSpan r = chunk_span<RT>(p, s, rt);
                const int n = r.hi / TK - r.lo / TK + 1;
                if (rem < n) {
                    start->t = r.lo / TK + int(rem);
                    break;
                }
                rem -= n;
            }
            start->b = b;
            start->g = g;
            start->rt = rt;
            start->item = w0;
            start->end = w1;
            start->total = total;
            break;
        }
    }
    __syncthreads();
}

template <int RT, int TK>
struct ChunkWalk {
    const ChunkParams& p;
    ChunkStart at;
    ChunkSeq s;
    int nrt;
    __device__ __forceinline__ ChunkWalk(const ChunkParams& pp, const ChunkStart& st) : p(pp), at(st) {
        if (at.item < at.end) {
            s = chunk_seq(p, at.b, false);
            nrt = chunk_row_tiles<RT>(p, s);
        }
    }
    // the next segment of this CTA, or false
    __device__ __forceinline__ bool next(ChunkSegment& seg) {
        if (at.item >= at.end) return false;
        seg.s = s;
        seg.span = chunk_span<RT>(p, s, at.rt);
        seg.b = at.b;
        seg.g = at.g;
        seg.rt = at.rt;
        seg.u0 = seg.span.lo / TK;
        seg.u1 = seg.span.hi / TK + 1;
        seg.t0 = at.t < 0 ? seg.u0 : at.t;
        seg.t1 = int(min(int64_t(seg.u1), seg.t0 + (at.end - at.item)));
        seg.item = at.item;
        at.item += seg.t1 - seg.t0;
        at.t = -1;
        if (++at.rt == nrt) {
            at.rt = 0;
            if (++at.g == p.hkv) {
                at.g = 0;
                if (at.item < at.end) {
                    do {
                        ++at.b;
                        s = chunk_seq(p, at.b, false);
                    } while (s.n == 0);
                    nrt = chunk_row_tiles<RT>(p, s);
                }
            }
        }
        return true;
    }
};

// Query row j's bit pattern or window, and whether it sees position u.
struct ChunkSight {
    int lo, hi;                // causal / window: positions [lo, hi]
    unsigned long long bits;   // tree: chunk positions
    int p0, n;
    bool tree;
    __device__ __forceinline__ bool sees(int u) const {
        if (!tree) return u >= lo && u <= hi;
        const int c = u - p0;
        return c < 0 || (c < n && ((bits >> c) & 1ull));
    }
};
__device__ __forceinline__ ChunkSight chunk_sight(const ChunkParams& p, const ChunkSeq& s, int j) {
    ChunkSight r;
    r.tree = p.tree != nullptr;
    r.p0 = s.p0;
    r.n = s.n;
    r.bits = r.tree ? __ldg(p.tree + s.row0 + j) : 0ull;
    r.hi = r.tree ? s.p0 + s.n - 1 : s.p0 + j;
    r.lo = !r.tree && p.window ? max(0, s.p0 + j + 1 - p.window) : 0;
    return r;
}

// The boxes of a segment's key tiles, 32 at a time, one per lane of the loading warp: box i holds positions
// i boxr .. + boxr - 1 (the tile in a contiguous cache, one block in a paged one; boxr = 2^box_log2).  A lane
// gives the first cache row, or -1 where no row of the row tile sees the box or its block is not valid
// (recorded).  The table is read two windows ahead of the tiles that use it: an entry takes about 2000 cycles
// to come from memory, longer than a tile.
struct ChunkBoxes {
    int base;        // first box of the window
    int row, next;   // this lane's box of the window and of the one behind it
    __device__ __forceinline__ int entry(const ChunkParams& p, const ChunkSegment& sg, int box) const {
        const int at = box << p.box_log2;
        if (at > sg.span.hi || at + (1 << p.box_log2) <= sg.span.lo) return -1;
        if (p.block_table == nullptr) return at;
        return __ldg(p.block_table + int64_t(sg.b) * p.mbps + (at >> p.bs_log2));
    }
    __device__ __forceinline__ int cache_row(const ChunkParams& p, const ChunkSegment& sg, int box, int e) const {
        const int at = box << p.box_log2;
        if (at > sg.span.hi || at + (1 << p.box_log2) <= sg.span.lo) return -1;
        if (p.block_table == nullptr) return (sg.b * p.hkv + sg.g) * p.capacity + at;
        if (e < 0 || e >= p.num_blocks) {
            record_status(YOCOPP_EDEVICE_CHECK);
            return -1;
        }
        return ((e * p.hkv + sg.g) << p.bs_log2) + (at & ((1 << p.bs_log2) - 1));
    }
    __device__ __forceinline__ void start(const ChunkParams& p, const ChunkSegment& sg, int box, int lane) {
        base = box & ~31;
        row = entry(p, sg, base + lane);
        next = entry(p, sg, base + 32 + lane);
        row = cache_row(p, sg, base + lane, row);
    }
    // the row of box `box + lane` for lane < n (n divides 32, box is a multiple of n), -1 in other lanes
    __device__ __forceinline__ int rows(const ChunkParams& p, const ChunkSegment& sg, int box, int n, int lane) {
        if (box >= base + 32) {
            base += 32;
            row = cache_row(p, sg, base + lane, next);
            next = entry(p, sg, base + 32 + lane);
        }
        const int r = __shfl_sync(0xffffffffu, row, (box - base + lane) & 31);
        return lane < n ? r : -1;
    }
};

// Slot of the workspace for a segment that is not a whole row tile: 0 where an earlier CTA began
// the row tile, 1 where this one did.
template <int RT, int D>
__device__ __forceinline__ float* chunk_slot(const ChunkParams& p, int cta, int which) {
    return p.part + (int64_t(cta) * 2 + which) * RT * (D + 2);
}

// Merge of the split row tiles: blocks (c, *) take the rows of the row tile that CTA c began and did not finish,
// if there is one: the parts are CTA c's slot 1 and slot 0 of the CTAs up to last_cta, merged exactly
// (out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i), D / 4 lanes a row, 8 parts in flight.  Bound by latency:
// the descriptor, the parts, and the instruction misses of code that runs once, so there is little of it.
constexpr int kChunkMergeThreads = 256, kChunkMergeFan = 4;
template <typename T, int D, int RT>
__global__ void __launch_bounds__(kChunkMergeThreads, 4) chunk_merge_kernel(const __grid_constant__ ChunkParams p) {
    constexpr int LPR = D / 4, ROWS = kChunkMergeThreads / LPR, F = kChunkMergeFan;
    const float ninf = __int_as_float(0xff800000);
    griddep_wait();
    const int c = blockIdx.x, ch = threadIdx.x % LPR;
    const int4 d = __ldcg(reinterpret_cast<const int4*>(p.desc + c));  // row0, first_row, rows, g
    const int last = __ldcg(&p.desc[c].last_cta);
    if (last < 0) return;
#pragma unroll 1
    for (int r = blockIdx.y * ROWS + threadIdx.x / LPR; r < d.z; r += gridDim.y * ROWS) {
        float M = ninf, L = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int i0 = c; i0 <= last; i0 += F) {
            float m[F], l[F];
            float4 x[F];
#pragma unroll
            for (int k = 0; k < F; ++k) {
                m[k] = ninf;
                if (i0 + k <= last) {
                    const float* s = chunk_slot<RT, D>(p, i0 + k, i0 + k == c ? 1 : 0);
                    m[k] = __ldcg(s + RT * D + r);
                    l[k] = __ldcg(s + RT * D + RT + r);
                    x[k] = __ldcg(reinterpret_cast<const float4*>(s + r * D) + ch);
                }
            }
            float mn = M;
#pragma unroll
            for (int k = 0; k < F; ++k) mn = fmaxf(mn, m[k]);
            if (mn == ninf) continue;  // parts in which the row sees nothing
            const float a = exp2f(M - mn);
            M = mn;
            L *= a;
            o = make_float4(o.x * a, o.y * a, o.z * a, o.w * a);
#pragma unroll
            for (int k = 0; k < F; ++k)
                if (m[k] != ninf) {
                    const float e = exp2f(m[k] - mn);
                    L = fmaf(l[k], e, L);
                    o = make_float4(fmaf(x[k].x, e, o.x), fmaf(x[k].y, e, o.y), fmaf(x[k].z, e, o.z), fmaf(x[k].w, e, o.w));
                }
        }
        const int row = d.y + r, j = chunk_token(p, row);
        const float inv = M == ninf ? 0.f : 1.f / L;
        T* out = reinterpret_cast<T*>(p.out) + ((int64_t(d.x) + j) * p.hq + d.w * p.G + (row - j * p.G)) * D + ch * 4;
        if constexpr (Elem<T>::kBytes == 2)
            *reinterpret_cast<uint2*>(out) = make_uint2(float2_to_bf16x2(o.x * inv, o.y * inv),
                                                        float2_to_bf16x2(o.z * inv, o.w * inv));
        else
            *reinterpret_cast<float4*>(out) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
}

}  // namespace yocopp
