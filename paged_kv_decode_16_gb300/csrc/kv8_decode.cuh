// kv8_decode.cuh -- decode attention over the 8-bit paged cache.
//
// As in the 16-bit kernel (schedule.cuh, decode_mma.cuh) a warp takes a
// balanced range of 16-token chunks through a ring of chunk buffers filled by
// tensor copies, and units spread over several warps leave fp32 partial states
// for a combine kernel.  A chunk is exactly one block of the cache, so it has
// one K scale 2^ek and one V scale 2^ev.  What differs: half the bytes a chunk
// leave half the time for everything beside them, so the ranges are worked out
// by every CTA for itself (no plan kernel before this one, for batches of up to
// kKv8SelfPlan sequences), they count a unit's start as kKv8UnitCost chunks
// more, a unit's queries are fetched while the unit before it is at work, and
// what is the same for a whole unit stays out of the loop over its chunks.
//
// Mathematics.  With x_t = (scale * log2 e) q.k8_t 2^ek(t) + ev(t), a running
// reference m and p_t = 2^(x_t - m):
//     o += p_t v8_t,   l += p_t 2^-ev(t),   out = o / l,
// since p_t v8_t = 2^(s_t - m) (v8_t 2^ev).  The V scale thus costs one add in
// the exponent, the largest p is about 1 whatever the scales are, and (m, l, o)
// merge like any other partial states.  (A term of l weighs 2^(s_t - m); a
// block whose p has left fp32's range, below 2^-126, still has no weight in l
// because the scales span at most 2^100.)  P is fp16, so m must suit the chunk at
// hand: a chunk whose ev lies far below the ones before it lowers m first (kKv8Span,
// kv8.cuh).
//
// Both products run transposed on m16n8k16 (fp16 in, fp32 accumulate), the 16
// tokens (S^T = K Q^T) or 16 elements of a head (O^T = V^T P^T) as the rows and
// 8 query rows as the columns: a GQA group of 4 to 8 fills a tile that would
// be half empty the other way round.  e4m3 is exact in fp16, so the cache
// enters without rounding.  bf16 queries are scaled by a power of two per row
// (largest element in [2^14, 2^15)) and are exact in fp16 down to 2^-31 of the
// row's largest element.  P is rounded to fp16 (11 bits), which is far below a bf16
// output's 8; for fp16 outputs what the rounding left enters in a second product
// (the error against 64 bits, 256 uneven sequences: 2.7e-4 of the norm without it,
// 2.1e-4 with it, which is the output's own rounding).
//
// The order of k in a product is free as long as both operands agree.  For
// S^T lane (j = lane / 4, t = lane % 4) takes D/4 consecutive elements of token
// j's row, for O^T D/8 consecutive elements of tokens 2t, 2t+1, 2t+8 and 2t+9:
// 16-byte shared loads straight from the copied rows, no transposing loads;
// with the copies' swizzle they hit every bank once (D = 64: V's twice).
//
// What bounds it: HBM for one query token a sequence -- 8 sequences of 32768
// tokens (537 MB): 83.4 us, 95% of the measured copy rate, and 5 more for the
// combine; 32 of 512 to 4096: 22 us of which about 4 are the start (the ranges, the
// page ids, the first copies, one after the other) and the uneven end, 77%.  About
// 330 instructions a chunk and warp (434 with the 16-bit kernel's chunk stream, 57 us
// for 8 sequences of 16384 against 50.2), 41% of the issue slots, 16% of the tensor
// pipe.  Units of 17 to 32 rows: the latency of their longer chunks at 8 warps an
// SM (5 query tokens, 20 rows: 46.5 us, 37% of HBM).
#pragma once

#include <cuda.h>

#include <type_traits>

#include "decode_mma.cuh"
#include "kv8_plan.cuh"
#include "merge.cuh"
#include "schedule.cuh"

namespace pkv {

// Positions.  Every unit (sequence, KV head, sub-group) with nch chunks has
// cost + nch positions, its chunks the last nch; all units' positions are laid
// end to end in unit order and cut into one range per worker, as in
// schedule.cuh.  prefix[b]: the first position of sequence b.
//
// Lane x holds the description of position 32 n + x of its worker's range, for
// the tile n that the consumer is in (a) and the next one (b), loaded a tile
// ahead so that no wait for it is in the loop.
struct Kv8Desc {
    int row;        // first pool row of the chunk; -1: nothing to copy
    uint32_t sc;    // its scales' bytes (K, V); bit 16 set: no tokens
    int u, k, len;  // unit, chunk of the unit (< 0: a cost position), tokens of the sequence
};

struct Kv8Stream {
    Kv8Desc a, b;
    int tile;  // tile of a
    int n;     // positions
    int f0, b_lo, b_hi, lane;
    uint32_t flags;  // PKV_DEV_* bits this lane has seen

    __device__ __forceinline__ Kv8Desc describe(const Kv8DecodeParams& p, const int32_t* prefix,
                                                int i) {
        Kv8Desc d = {-1, 1u << 16, 0, 0, 0};
        if (i >= n) return d;
        const int f = f0 + i;
        int lo = b_lo, hi = b_hi;  // the last sequence with prefix <= f: empty ones are passed over
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (prefix[mid] <= f) lo = mid; else hi = mid;
        }
        const int first = prefix[lo];
        const int per_unit = (prefix[lo + 1] - first) / p.units_per_b;
        const int rem = f - first;
        const int uidx = rem / per_unit;
        d.u = lo * p.units_per_b + uidx;
        d.k = rem - uidx * per_unit - p.unit_cost;
        d.len = (int)min((long long)p.lens[lo], p.cap);
        if (d.k < 0) return d;
        const int col = kv8_page_col(d.k, p.page_magic);
        const int page = __ldg(p.table + (long long)lo * p.table_stride + col);
        if (page >= 0 && page < p.num_pages) {
            const int blk = (page * p.n_kv_heads + uidx / p.sub_groups) * p.chunks_per_page +
                            (d.k - col * p.chunks_per_page);
            d.row = blk * kChunk;  // below 2^31: checked on the host
            d.sc = (uint32_t)p.scales[blk];  // (an append may write it before the wait)
        } else {
            flags |= PKV_DEV_BAD_PAGE;
        }
        return d;
    }
    __device__ __forceinline__ void next(const Kv8DecodeParams& p, const int32_t* prefix) {
        b = describe(p, prefix, (tile + 1) * 32 + lane);
    }
    // The consumer has come to position i; true: into a new tile.
    __device__ __forceinline__ bool advance(const Kv8DecodeParams& p, const int32_t* prefix,
                                            int i) {
        if ((i >> 5) == tile) return false;
        a = b;
        ++tile;
        next(p, prefix);
        return true;
    }
    // Row, unit of position i (in tile a or b); the scales of one in tile a.
    __device__ __forceinline__ int row(int i) const {
        const int v = (i >> 5) == tile ? a.row : b.row;
        return __shfl_sync(kFull, v, i & 31);
    }
    __device__ __forceinline__ int unit(int i) const {
        const int v = (i >> 5) == tile ? a.u : b.u;
        return __shfl_sync(kFull, v, i & 31);
    }
    __device__ __forceinline__ uint32_t sc(int i) const { return __shfl_sync(kFull, a.sc, i & 31); }
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The 8x8 matrix of 16-bit elements held one row a quad, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

// Bit 7 of every byte that is an e4m3 NaN (0x7f or 0xff).
__device__ __forceinline__ uint32_t e4m3_nan_mask(uint32_t w) {
    return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// Shared memory of one CTA: every warp's ring of chunks (K then V), its next
// unit's query rows as they come (units of up to 16 rows), the query fragments
// (larger units), the mbarriers, and the plan's prefix sums.
template <int D, int NT, int STAGES, int WARPS>
struct Kv8Layout {
    static constexpr int kSide = kChunk * D;  // K or V bytes of a chunk
    static constexpr int kStageBytes = 2 * kSide;
    static constexpr int kWarpKV = STAGES * kStageBytes;
    static constexpr bool kQShared = NT > 2;
    static constexpr int kWarpQ = NT * 8 * D * 2;
    static constexpr int kOffQ = WARPS * kWarpKV;
    static constexpr int kOffBar = kOffQ + WARPS * kWarpQ;
    static constexpr int kOffPlan = kOffBar + WARPS * STAGES * 8;
    static constexpr int kBytes = kOffPlan + (kKv8SelfPlan + 1) * 4 + 1024;  // + alignment slack
};

// NT tiles of 8 query rows; a unit has at most 8 NT rows.
template <typename T, int D, int NT, int WARPS, int STAGES, int CTAS>
__global__ void __launch_bounds__(WARPS * 32, CTAS)
kv8_decode_kernel(const __grid_constant__ Kv8DecodeParams p,
                  const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
    using Lay = Kv8Layout<D, NT, STAGES, WARPS>;
    constexpr int KSTEPS = D / 16;  // k-steps of S^T
    constexpr int MT = D / 16;      // m16 tiles of O^T
    constexpr int DPL = D / 8;      // V elements a lane takes of a row
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr bool kSplitP = !kBf16;  // P in two fp16 pieces

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;  // the swizzle's period
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    uint8_t* base = smem_raw + pad;
    uint8_t* wsm = base + warp * Lay::kWarpKV;
    const uint32_t wsm_u32 = raw + pad + warp * Lay::kWarpKV;
    // query rows: 16-byte vector x of tile n at (n * KSTEPS / 2 + x) * 512 + lane * 16
    const uint32_t sq = raw + pad + Lay::kOffQ + warp * Lay::kWarpQ + lane * 16;
    uint64_t* bar = reinterpret_cast<uint64_t*>(base + Lay::kOffBar) + warp * STAGES;
    int32_t* s_prefix = reinterpret_cast<int32_t*>(base + Lay::kOffPlan);

    // every warp's last segment, when it holds a part of a unit: the unit (-1:
    // none), whether it has the unit's first (1) and last (2) chunk, and its
    // rows' maxima and sums (its weighted sums take the place of the ring)
    struct Tail {
        int u, ends, b, h, sg, rows;
    };
    __shared__ Tail s_tail[WARPS];
    __shared__ float s_ml[WARPS][2 * 8 * NT];
    static_assert(NT * 8 * D * 4 <= Lay::kWarpKV, "a segment's sums fit its ring");

    if (lane == 0) {
        s_tail[warp].u = -1;
#pragma unroll
        for (int s = 0; s < STAGES; ++s) mbar_init(&bar[s], 1);
        fence_barrier_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap))
                     : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap))
                     : "memory");
    }
    __syncwarp();
    // After a step's append the ranges are worked out beside it: that kernel lets
    // this one start only after its own wait, so every kernel before it is
    // complete, and it writes neither the lengths nor the ranges' place in the
    // workspace.  (The rows, scales and rotated queries it does write: below the
    // wait.)
    const bool early = p.after_append && p.self_plan;
    if (!early) pdl_wait();

    const int gw = blockIdx.x * WARPS + warp;
    Kv8Stream ws;
    ws.flags = 0;
    ws.lane = lane;
    ws.tile = 0;
    ws.b_lo = 0;
    ws.b_hi = p.batch;
    const int32_t* prefix;
    int nw, sw, r;
    if (p.self_plan) {
        const int total = kv8_self_plan<WARPS * 32>(p, s_prefix, &ws.flags);
        prefix = s_prefix;
        kv8_ranges(total, p.workers_req, p.workers_auto, &nw, &sw, &r);
        if (gw == 0 && lane == 0) {
            p.hdr->num_workers = nw;
            p.hdr->chunks_per_worker = sw;
            p.hdr->extra_chunks = r;
        }
    } else {
        prefix = p.prefix;
        nw = p.hdr->num_workers;
        sw = p.hdr->chunks_per_worker;
        r = p.hdr->extra_chunks;
    }
    if (early) pdl_wait();
    const int merge_warps = kv8_merge_warps(p.units, nw, p.merge);
    ws.f0 = range_begin(gw, sw, r);
    ws.n = gw < nw ? sw + (gw < r ? 1 : 0) : 0;
    ws.a = ws.describe(p, prefix, lane);

    const uint64_t kv_policy = l2_evict_first_policy();
    const int j = lane >> 2, t = lane & 3;

    // Copy the chunk of position i into stage st.
    auto issue = [&](int i, int st) {
        const int row = ws.row(i);
        if (lane == 0) {
            uint64_t* bp = &bar[st];
            uint8_t* dst = wsm + st * Lay::kStageBytes;
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(bp, row >= 0 ? (uint32_t)Lay::kStageBytes : 0u);
            if (row >= 0) {
                tma_load_2d_hint(dst, &kmap, 0, row, bp, kv_policy);
                tma_load_2d_hint(dst + Lay::kSide, &vmap, 0, row, bp, kv_policy);
            }
        }
    };
    // Fetch this lane's part of the query rows of the unit of position i (its
    // own 16-byte vectors only, so only this lane waits for them).
    auto fetch_q = [&](int i) {
        const int u = ws.unit(i);
        const int b = u / p.units_per_b;
        const int uidx = u - b * p.units_per_b;
        const int h = uidx / p.sub_groups;
        const int sg = uidx - h * p.sub_groups;
        const int rows = p.rows.rows(sg);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            // lane (j, t) takes elements D/4 t .. of row 8n + j
            const int rr = 8 * n + j;
            const bool ok = rr < rows;
            const T* src = static_cast<const T*>(p.q) +
                           (ok ? p.rows.row(b, h, sg, rr) * D : 0) + t * (D / 4);
#pragma unroll
            for (int x = 0; x < KSTEPS / 2; ++x)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                                 sq + (n * (KSTEPS / 2) + x) * 512),
                             "l"(src + x * 8), "r"(ok ? 16 : 0)
                             : "memory");
        }
    };

    if (ws.n > 0) {
#pragma unroll
        for (int s = 0; s < STAGES; ++s)
            if (s < ws.n) issue(s, s);
        fetch_q(0);
        ws.next(p, prefix);  // the second tile, behind the first copies
    }
    // rows of sequences with no tokens are zeros: no worker visits them (nor, when
    // the positions are too many and nothing is done, any)
    for (int b = gw; b < p.batch; b += gridDim.x * WARPS) {
        if (prefix[b] != prefix[b + 1] && nw > 0) continue;
        const long long vecs = (long long)p.rows.n_queries * p.rows.n_q_heads * D / 8;
        uint4* dst = reinterpret_cast<uint4*>(p.out) + b * vecs;
        for (long long x = lane; x < vecs; x += 32) dst[x] = make_uint4(0u, 0u, 0u, 0u);
    }

    int st = 0;          // stage of the position at hand
    uint32_t phase = 0;  // its barrier's phase
    int i = 0;           // position
    bool q_coming = true;  // the next unit's query rows are on the way
    // a position is done with: its stage takes the one STAGES further on
    auto release = [&](int pos) {
        __syncwarp();
        if (pos + STAGES < ws.n) issue(pos + STAGES, st);
        if (++st == STAGES) {
            st = 0;
            phase ^= 1u;
        }
    };
    while (i < ws.n) {
        // ---- a segment: the positions of one unit in this range ----
        ws.advance(p, prefix, i);
        const int u = __shfl_sync(kFull, ws.a.u, i & 31);
        int k0 = __shfl_sync(kFull, ws.a.k, i & 31);
        const int len = __shfl_sync(kFull, ws.a.len, i & 31);
        const int nch = len / kChunk + (len % kChunk != 0);  // (len + 15 may pass 32 bits)
        if (!q_coming) fetch_q(i);
        const int end = i + min(nch - k0, ws.n - i);
        for (; k0 < 0 && i < end; ++i, ++k0) release(i);  // cost positions hold nothing
        const int b = u / p.units_per_b;
        const int uidx = u - b * p.units_per_b;
        const int h = uidx / p.sub_groups;
        const int sg = uidx - h * p.sub_groups;
        const int rows = p.rows.rows(sg);
        const int last = len - p.rows.n_queries;            // last token that query 0 sees
        const int lim_min = last + p.rows.first_query(sg);  // the unit's first row's

        uint32_t qf[Lay::kQShared ? 1 : NT][KSTEPS][2];  // B fragments of Q^T
        float fs[NT][2];  // score factors of rows 2t, 2t+1 of a tile: scale log2(e) / row scale
        float o[NT][MT][4];  // O^T: elements DPL j + 2i (c0, c1), + 1 (c2, c3) of rows 2t, 2t+1
        // reference of rows 2t, 2t+1; the same with 0 for -inf, less kKv8Lift (after a
        // range's first chunk the accumulators are hardly ever rescaled: kKv8Slack)
        float m[NT][2], mr[NT][2];
        float l[NT][2];           // this lane's part of the rows' sums
        int ev_ref = kKv8MinExp;  // the V exponent that the references suit
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            uint32_t x4[KSTEPS * 2];
#pragma unroll
            for (int x = 0; x < KSTEPS / 2; ++x) {
                const uint4 v = lds128(sq + (n * (KSTEPS / 2) + x) * 512);
                x4[4 * x] = v.x;
                x4[4 * x + 1] = v.y;
                x4[4 * x + 2] = v.z;
                x4[4 * x + 3] = v.w;
            }
            int shift = 0;  // the row is multiplied by 2^shift
            if constexpr (kBf16) {
                uint32_t mx = 0u;
#pragma unroll
                for (int x = 0; x < KSTEPS * 2; ++x) mx = __vmaxu2(mx, x4[x] & 0x7fff7fffu);
                mx = max(mx & 0xffffu, mx >> 16);
                mx = max(mx, __shfl_xor_sync(kFull, mx, 1));
                mx = max(mx, __shfl_xor_sync(kFull, mx, 2));
                shift = mx == 0u ? 0 : min(141 - (int)(mx >> 7), 126);
                const float f = exp2i(shift);
#pragma unroll
                for (int x = 0; x < KSTEPS * 2; ++x)
                    x4[x] = Cvt<__half>::pack2(__uint_as_float(x4[x] << 16) * f,
                                               __uint_as_float(x4[x] & 0xffff0000u) * f);
            }
            if constexpr (Lay::kQShared) {
                if constexpr (kBf16) {
#pragma unroll
                    for (int x = 0; x < KSTEPS / 2; ++x)
                        sts128(sq + (n * (KSTEPS / 2) + x) * 512,
                               make_uint4(x4[4 * x], x4[4 * x + 1], x4[4 * x + 2], x4[4 * x + 3]));
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < KSTEPS; ++kk) {
                    qf[n][kk][0] = x4[2 * kk];
                    qf[n][kk][1] = x4[2 * kk + 1];
                }
            }
            // factors of the rows this lane's accumulators hold
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int sh = __shfl_sync(kFull, shift, 4 * (2 * t + c));
                fs[n][c] = p.scale_log2 * exp2i(-sh);
                m[n][c] = -INFINITY;
                mr[n][c] = 0.f;
                l[n][c] = 0.f;
            }
#pragma unroll
            for (int x = 0; x < MT; ++x) o[n][x][0] = o[n][x][1] = o[n][x][2] = o[n][x][3] = 0.f;
        }
        // the buffer is free again (larger units keep their fragments in it)
        q_coming = !Lay::kQShared && end < ws.n && (end >> 5) <= ws.tile + 1;
        if (q_coming) fetch_q(end);

        for (int pos = i; pos < end; ++pos) {
            if (ws.advance(p, prefix, pos) && !Lay::kQShared && !q_coming && end < ws.n &&
                (end >> 5) <= ws.tile + 1) {
                fetch_q(end);
                q_coming = true;
            }
            if (!mbar_wait_bounded(&bar[st], phase)) {
                ws.flags |= PKV_DEV_TIMEOUT;
                // wait (bounded) for the copies still in flight into this warp's buffers
                for (int s = 1; s < STAGES; ++s) {
                    const int s2 = (st + s) % STAGES;
                    if (pos + s < ws.n) mbar_wait_bounded(&bar[s2], s2 > st ? phase : phase ^ 1u);
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                ws.n = 0;
                break;
            }
            const int tok0 = (k0 + pos - i) * kChunk;  // the chunk's first token
            const uint32_t sc = ws.sc(pos);
            const float fk = __uint_as_float((sc & 0xffu) << 23);  // 2^ek (byte 0: 0)
            const int evi = kv8_clamp_exp((int)((sc >> 8) & 0xffu) - 127);
            const float ev = (float)evi, inv_v = exp2i(-evi);
            const bool low = evi < ev_ref - kKv8Span;
            ev_ref = low ? evi : max(ev_ref, evi);
            const int nv = (sc >> 16) ? 0 : min(kChunk, len - tok0);  // tokens that count
            // rows see every token of the chunk, or masks apply
            const bool masked = nv < kChunk || tok0 + kChunk - 1 > lim_min;
            const uint32_t kst = wsm_u32 + st * Lay::kStageBytes;
            const uint32_t vst = kst + Lay::kSide;
            // ---- S^T = K Q^T ----
            float s[NT][4];
            {
                uint32_t kw[2][KSTEPS];  // token rows j and j + 8: D/4 bytes each
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const int row = j + 8 * hf;
                    if constexpr (D == 128) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint4 v =
                                lds128(kst + row * 128 + (((2 * t + x) ^ (row & 7)) << 4));
                            kw[hf][4 * x] = v.x;
                            kw[hf][4 * x + 1] = v.y;
                            kw[hf][4 * x + 2] = v.z;
                            kw[hf][4 * x + 3] = v.w;
                        }
                    } else {
                        const uint4 v = lds128(kst + row * 64 + ((t ^ ((row >> 1) & 3)) << 4));
                        kw[hf][0] = v.x;
                        kw[hf][1] = v.y;
                        kw[hf][2] = v.z;
                        kw[hf][3] = v.w;
                    }
                }
                // one unit tile: two chains of products, added at the end
                constexpr int KC = NT == 1 ? 2 : 1;
                float sk[NT][KC][4];
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < KC; ++c)
                        sk[n][c][0] = sk[n][c][1] = sk[n][c][2] = sk[n][c][3] = 0.f;
#pragma unroll
                for (int kk = 0; kk < KSTEPS; kk += 2) {
                    uint32_t a[2][4];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        e4m3x4_to_h2(kw[0][kk + x], a[x][0], a[x][2]);
                        e4m3x4_to_h2(kw[1][kk + x], a[x][1], a[x][3]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if constexpr (Lay::kQShared) {
                            const uint4 q4 = lds128(sq + (n * (KSTEPS / 2) + kk / 2) * 512);
                            mma_f16(sk[n][0], a[0][0], a[0][1], a[0][2], a[0][3], q4.x, q4.y);
                            mma_f16(sk[n][KC - 1], a[1][0], a[1][1], a[1][2], a[1][3], q4.z, q4.w);
                        } else {
                            mma_f16(sk[n][0], a[0][0], a[0][1], a[0][2], a[0][3], qf[n][kk][0],
                                    qf[n][kk][1]);
                            mma_f16(sk[n][KC - 1], a[1][0], a[1][1], a[1][2], a[1][3],
                                    qf[n][kk + 1][0], qf[n][kk + 1][1]);
                        }
                    }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        s[n][e] = KC == 1 ? sk[n][0][e] : sk[n][0][e] + sk[n][KC - 1][e];
            }
            // ---- exponents ----
            bool above = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[n][e] = fmaf(s[n][e], fs[n][e & 1] * fk, ev);
                    if (masked) {
                        const int tok = j + 8 * (e >> 1);
                        const int lim = last + p.rows.query(sg, 8 * n + 2 * t + (e & 1));
                        if (tok >= nv || tok0 + tok > lim) s[n][e] = -INFINITY;
                    }
                    top[e & 1] = fmaxf(top[e & 1], s[n][e]);
                }
                above |= top[0] > m[n][0] + kKv8Slack || top[1] > m[n][1] + kKv8Slack;
            }
            if (__any_sync(kFull, above || low)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = fmaxf(s[n][c], s[n][c + 2]);
                        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
                        float m_new = fmaxf(m[n][c], mx);
                        if (low) {  // down to what suits the row's sum so far
                            float lr = l[n][c];
                            lr += __shfl_xor_sync(kFull, lr, 4);
                            lr += __shfl_xor_sync(kFull, lr, 8);
                            lr += __shfl_xor_sync(kFull, lr, 16);
                            m_new = fminf(m_new, fmaxf(mx, __log2f(lr) + mr[n][c] + ev));
                        }
                        // a row that has seen no token yet: reference 0, weights 0
                        const float ref = m_new == -INFINITY ? 0.f : m_new;
                        mr[n][c] = ref - kKv8Lift;
                        const float alpha = fast_exp2(m[n][c] - ref);
                        m[n][c] = m_new;
                        l[n][c] *= alpha;
#pragma unroll
                        for (int x = 0; x < MT; ++x) {
                            o[n][x][c] *= alpha;
                            o[n][x][c + 2] *= alpha;
                        }
                    }
            }
            {
                uint32_t pb[NT][2];  // B fragments of P^T: tokens 2t, 2t+1 (+ 8) of row j
                uint32_t pl[NT][2];  // fp16 outputs: what P's rounding left
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const float p0 = fast_exp2(s[n][0] - mr[n][0]);
                    const float p1 = fast_exp2(s[n][1] - mr[n][1]);
                    const float p2 = fast_exp2(s[n][2] - mr[n][0]);
                    const float p3 = fast_exp2(s[n][3] - mr[n][1]);
                    l[n][0] = fmaf(p0 + p2, inv_v, l[n][0]);
                    l[n][1] = fmaf(p1 + p3, inv_v, l[n][1]);
                    const uint32_t h0 = Cvt<__half>::pack2(p0, p1);
                    const uint32_t h1 = Cvt<__half>::pack2(p2, p3);
                    pb[n][0] = transpose8x8(h0);
                    pb[n][1] = transpose8x8(h1);
                    if constexpr (kSplitP) {
                        const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
                        const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
                        pl[n][0] = transpose8x8(Cvt<__half>::pack2(p0 - f0.x, p1 - f0.y));
                        pl[n][1] = transpose8x8(Cvt<__half>::pack2(p2 - f1.x, p3 - f1.y));
                    }
                }
                // ---- O^T += V^T P^T ----
                uint32_t vw[4][DPL / 4];  // tokens 2t, 2t+1, 2t+8, 2t+9: elements DPL j ..
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int row = 2 * t + (x & 1) + 8 * (x >> 1);
                    if constexpr (D == 128) {
                        const uint4 v = lds128(vst + row * 128 + ((j ^ (row & 7)) << 4));
                        vw[x][0] = v.x;
                        vw[x][1] = v.y;
                        vw[x][2] = v.z;
                        vw[x][3] = v.w;
                    } else {
                        const uint32_t addr =
                            vst + row * 64 + (((j >> 1) ^ ((row >> 1) & 3)) << 4) + (j & 1) * 8;
                        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                     : "=r"(vw[x][0]), "=r"(vw[x][1])
                                     : "r"(addr));
                    }
                }
                // A NaN in V at a token that some row does not see must not
                // reach that row through its weight 0: such a chunk (a block
                // behind the sequence's end may hold anything) multiplies with
                // the NaNs taken out and adds them back for the rows that see
                // them.
                if (masked) {
                    uint32_t any = 0u;
#pragma unroll
                    for (int x = 0; x < 4; ++x)
#pragma unroll
                        for (int w = 0; w < DPL / 4; ++w) any |= e4m3_nan_mask(vw[x][w]);
                    if (__any_sync(kFull, any != 0u)) {
#pragma unroll
                        for (int w = 0; w < DPL / 4; ++w) {
                            uint32_t nan[4];
#pragma unroll
                            for (int x = 0; x < 4; ++x) {
                                nan[x] = e4m3_nan_mask(vw[x][w]) >> 7;  // 1 in each NaN's byte
                                vw[x][w] &= ~(nan[x] * 0xffu);
                                nan[x] *= 0x38u;  // 1.0
                            }
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const uint32_t sel = hf == 0 ? 0x5140u : 0x7362u;
                                uint32_t a0, a1, a2, a3;
                                e4m3x4_to_h2(__byte_perm(nan[0], nan[1], sel), a0, a1);
                                e4m3x4_to_h2(__byte_perm(nan[2], nan[3], sel), a2, a3);
#pragma unroll
                                for (int n = 0; n < NT; ++n) {
                                    // the last token of the chunk that row 8n + j sees
                                    const int lr =
                                        min(last + p.rows.query(sg, 8 * n + j) - tok0,
                                            nv - 1);
                                    const uint32_t v0 = (2 * t <= lr ? 0x3c00u : 0u) |
                                                        (2 * t + 1 <= lr ? 0x3c000000u : 0u);
                                    const uint32_t v1 = (2 * t + 8 <= lr ? 0x3c00u : 0u) |
                                                        (2 * t + 9 <= lr ? 0x3c000000u : 0u);
                                    float c4[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma_f16(c4, a0, a1, a2, a3, v0, v1);
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        if (c4[e] > 0.f)
                                            o[n][2 * w + hf][e] = __uint_as_float(0x7fc00000u);
                                }
                            }
                        }
                    }
                }
#pragma unroll
                for (int w = 0; w < DPL / 4; ++w) {
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        const uint32_t sel = hf == 0 ? 0x5140u : 0x7362u;
                        uint32_t a0, a1, a2, a3;
                        e4m3x4_to_h2(__byte_perm(vw[0][w], vw[1][w], sel), a0, a1);
                        e4m3x4_to_h2(__byte_perm(vw[2][w], vw[3][w], sel), a2, a3);
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            mma_f16(o[n][2 * w + hf], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                        if constexpr (kSplitP) {
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma_f16(o[n][2 * w + hf], a0, a1, a2, a3, pl[n][0], pl[n][1]);
                        }
                    }
                }
            }
            release(pos);
        }
        if (ws.n == 0) break;  // gave up

        // ---- the segment's result ----
        // the whole unit: its output; a part: a partial state -- except, with
        // merge_warps, where the range ends within the unit or with it: to
        // shared memory, merged below with the other warps' of the CTA
        const bool whole = k0 == 0 && end - i == nch;
        const bool to_tail = !whole && end == ws.n && merge_warps > 1;
        if (to_tail && i < end && lane == 0) {
            s_tail[warp] = {u, (k0 == 0 ? 1 : 0) | (k0 + end - i == nch ? 2 : 0), b, h, sg, rows};
        }
        float* slot = p.partials + (long long)(u + gw) * partial_slot_floats(p.gs, D);
        float* sm_o = reinterpret_cast<float*>(wsm);  // the ring: its copies are all used up
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                if (i == end) continue;  // cost positions only
                float lr = l[n][c];
                lr += __shfl_xor_sync(kFull, lr, 4);
                lr += __shfl_xor_sync(kFull, lr, 8);
                lr += __shfl_xor_sync(kFull, lr, 16);
                const int r = 8 * n + 2 * t + c;
                if (r >= rows) continue;
                if (whole) {
                    const float inv = lr == 0.f ? 0.f : 1.0f / lr;  // no token seen: zeros
                    uint4* dst = reinterpret_cast<uint4*>(
                        static_cast<T*>(p.out) + p.rows.row(b, h, sg, r) * D + DPL * j);
#pragma unroll
                    for (int x = 0; x < MT / 4; ++x)
                        dst[x] = make_uint4(
                            Cvt<T>::pack2(o[n][4 * x][c] * inv, o[n][4 * x][c + 2] * inv),
                            Cvt<T>::pack2(o[n][4 * x + 1][c] * inv, o[n][4 * x + 1][c + 2] * inv),
                            Cvt<T>::pack2(o[n][4 * x + 2][c] * inv, o[n][4 * x + 2][c + 2] * inv),
                            Cvt<T>::pack2(o[n][4 * x + 3][c] * inv, o[n][4 * x + 3][c + 2] * inv));
                } else {
                    float4* dst =
                        reinterpret_cast<float4*>((to_tail ? sm_o : slot) + r * D + DPL * j);
#pragma unroll
                    for (int x = 0; x < MT / 2; ++x)
                        dst[x] = make_float4(o[n][2 * x][c], o[n][2 * x][c + 2],
                                             o[n][2 * x + 1][c], o[n][2 * x + 1][c + 2]);
                    if (j == 0) {
                        float* ml = to_tail ? s_ml[warp] : slot + p.gs * D;
                        ml[r] = m[n][c];
                        ml[(to_tail ? 8 * NT : p.gs) + r] = lr;
                    }
                }
            }
        i = end;
    }
    const uint32_t flags = __reduce_or_sync(kFull, ws.flags);
    if (lane == 0) p.flags[gw] = flags;
    if (merge_warps == 1) {
        pdl_trigger();
        return;
    }
    __syncthreads();

    // ---- the warps' last segments: neighbours of one unit become one state ----
    int tail_u[WARPS];
#pragma unroll
    for (int w = 0; w < WARPS; ++w) tail_u[w] = s_tail[w].u;
#pragma unroll
    for (int w0 = 0; w0 < WARPS; ++w0) {
        const int u = tail_u[w0];
        if (u < 0 || (w0 > 0 && tail_u[w0 > 0 ? w0 - 1 : 0] == u)) continue;
        int w1 = w0 + 1;
#pragma unroll
        for (int w = w0 + 1; w < WARPS; ++w)
            if (w1 == w && tail_u[w] == u) w1 = w + 1;
        const bool whole = (s_tail[w0].ends & 1) && (s_tail[w1 - 1].ends & 2);
        const int b = s_tail[w0].b, h = s_tail[w0].h, sg = s_tail[w0].sg;
        const int rows = s_tail[w0].rows;
        float* slot = p.partials + (long long)(u + blockIdx.x * WARPS + w0) *
                                       partial_slot_floats(p.gs, D);
        for (int x = threadIdx.x; x < rows * (D / 4); x += WARPS * 32) {
            const int r = x / (D / 4), v = x - r * (D / 4);
            float M = -INFINITY;
            for (int w = w0; w < w1; ++w) M = fmaxf(M, s_ml[w][r]);
            float den = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = w0; w < w1; ++w) {
                const float wt = merge_weight(s_ml[w][r], M);
                const float4 y =
                    reinterpret_cast<const float4*>(base + w * Lay::kWarpKV)[r * (D / 4) + v];
                den = fmaf(wt, s_ml[w][8 * NT + r], den);
                acc.x = fmaf(wt, y.x, acc.x);
                acc.y = fmaf(wt, y.y, acc.y);
                acc.z = fmaf(wt, y.z, acc.z);
                acc.w = fmaf(wt, y.w, acc.w);
            }
            if (whole) {
                const float inv = den == 0.f ? 0.f : 1.0f / den;
                *reinterpret_cast<uint2*>(static_cast<T*>(p.out) +
                                          p.rows.row(b, h, sg, r) * D + 4 * v) =
                    make_uint2(Cvt<T>::pack2(acc.x * inv, acc.y * inv),
                               Cvt<T>::pack2(acc.z * inv, acc.w * inv));
            } else {
                reinterpret_cast<float4*>(slot + r * D)[v] = acc;
                if (v == 0) {
                    slot[p.gs * D + r] = M;
                    slot[p.gs * D + p.gs + r] = den;
                }
            }
        }
    }
    pdl_trigger();
}

template <typename T, int D, int NT>
Kv8DecodeInfo make_kv8_decode_info() {
    // Chunks on the way: one tile of rows, 12 warps of 2 stages (96 KiB an SM; 3
    // stages took 93.1 us of 8 sequences of 32768 tokens, 4 took 97.0, 2 take 90.4:
    // more copies in flight than the memory needs cost it order).  Larger units hold
    // their accumulators in all the registers that 8 warps leave (3 CTAs of fewer
    // registers, or 2 warps a CTA, spill: 69 us against 45 of 5 query tokens).
    constexpr int W = kKv8Warps, S = NT == 1 ? 2 : NT == 3 ? 3 : 4, C = NT == 1 ? 3 : 2;
    Kv8DecodeInfo info;
    info.fn = kv8_decode_kernel<T, D, NT, W, S, C>;
    info.warps = W;
    info.threads = W * 32;
    info.smem_bytes = Kv8Layout<D, NT, S, W>::kBytes;
    return info;
}

template <typename T>
Kv8DecodeInfo pick_kv8_decode_info(int head_dim, int rows) {
    if (head_dim == 128)
        return rows <= 8    ? make_kv8_decode_info<T, 128, 1>()
               : rows <= 16 ? make_kv8_decode_info<T, 128, 2>()
               : rows <= 24 ? make_kv8_decode_info<T, 128, 3>()
                            : make_kv8_decode_info<T, 128, 4>();
    return rows <= 8    ? make_kv8_decode_info<T, 64, 1>()
           : rows <= 16 ? make_kv8_decode_info<T, 64, 2>()
           : rows <= 24 ? make_kv8_decode_info<T, 64, 3>()
                        : make_kv8_decode_info<T, 64, 4>();
}

}  // namespace pkv
