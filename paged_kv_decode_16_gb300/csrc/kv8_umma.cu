// kv8_umma.cu -- attention of many query rows over the 8-bit paged cache on the
// fifth-generation tensor cores (tcgen05, accumulators in tensor memory).
//
// For several query tokens a sequence whose rows (tokens x heads of the GQA
// group) fill a good part of a 128-row tile.  The mathematics is kv8_decode.cuh's
// (one exponent for the weights and the V scales); a unit is up to 128 rows, a
// worker a CTA, and a CTA's range is walked in blocks of up to 8 chunks (128
// tokens):
//
//   S = Q K^T         M = 128 rows, N = tokens, K = D   (fp16, fp32 accumulate)
//   P = 2^(x - m)     two threads a row, half of the tokens each
//   O = O 2^(m_old - m) + P V     M = 128, N = D, K = tokens
//
// A block with a V exponent too far from those before it (kKv8Span, kv8.cuh) takes
// the last two steps a chunk at a time, each with a reference that suits it.
//
// The e4m3 bytes come by 16-byte loads from L2 into registers, a warp a chunk (its
// page, scales and length are then the warp's), K's during the softmax of the block
// before and V's during its last product.  They are converted to fp16, which holds
// them exactly, and stored in the 128-byte swizzled layout that the tensor cores
// read; K's place takes P once S is done, so that two CTAs share an SM and one's
// products run under the other's conversion and softmax.  (No place is left for what
// P's rounding to fp16 leaves, which the warp kernel takes along for fp16 outputs: 64
// query tokens' error against 64 bits is 2.7e-4 of the norm, there 2.1e-4.)  (Tensor copies would
// need 32 KiB more for the raw bytes, and leave one CTA an SM.)
//
// What bounds it: the chain of a block's phases -- convert, product, maximum,
// exponentials, product, with a barrier or a wait between them -- of about 8000
// cycles, of which two CTAs an SM overlap; the floor beneath is 1024 cycles of
// exponentials (16 a cycle and SM) and as many of products for a block of 128 x
// 128.  4 sequences of 1000 to 8192 tokens with 64 query tokens, 32/8 heads of 128:
// 54.3 us with the combine (294 TFLOP/s), against 107 on the warp kernel; the issue
// slots are 40% busy, the tensor pipe 15%.
//
// Every wait is bounded: on a timeout the CTA reports PKV_DEV_TIMEOUT, waits
// (bounded) once more for its products in flight, frees its tensor memory and
// returns.
#include <type_traits>

#include "kv8_plan.cuh"
#include "umma.cuh"

namespace pkv {

namespace {

constexpr int kRows = kKv8UmmaRows;   // M: one tensor-memory lane a row
constexpr int kBlockChunks = 8;
constexpr int kBlockTok = kBlockChunks * kChunk;
// (Four threads a row, in 64 registers each, spill: 86 against 63 us.)
constexpr int kThreads = 256;
constexpr int kNoExp = -100;  // below every exponent: no chunk, or none with tokens yet
constexpr int kParts = kThreads / 128;             // threads a row: each its part of the tokens
constexpr int kPartChunks = kBlockChunks / kParts;  // ... and of O's columns

// Shared memory of one CTA from a 1 KiB aligned base: fp16 column blocks of 64
// elements (128 bytes a row), 8-row groups of 1 KiB.
template <int D>
struct Layout {
    static constexpr int kCols = D / 64;
    static constexpr int kColBytes = 128 * 128;  // a column block of 128 rows
    static constexpr int kOffQ = 0;
    static constexpr int kOffK = kOffQ + kCols * kColBytes;  // K, then P (2 blocks of 64 tokens)
    static constexpr int kOffV = kOffK + 2 * kColBytes;
    static constexpr int kOffEnd = kOffV + kCols * kColBytes;
    static constexpr int kOffMax = kOffEnd;                  // [parts][128] floats
    static constexpr int kOffChunk = kOffMax + kParts * 128 * 4;  // [8] ChunkInfo
    static constexpr int kOffEv = kOffChunk + kBlockChunks * 16;  // [8] V exponents, a byte each
    static constexpr int kOffBar = kOffEv + kBlockChunks;
    static constexpr int kOffPlan = kOffBar + 32;
    static constexpr int kUsed = kOffPlan + (kKv8SelfPlan + 1) * 4 + 1024;
    // at least 80 KiB: no more CTAs on an SM than its tensor memory serves
    static constexpr int kBytes = kUsed > 80 * 1024 ? kUsed : 80 * 1024;
    static constexpr int kColsS = kBlockTok;  // tensor memory: S, then O
    static constexpr int kTmemCols = 256;
    static_assert(kColsS + D <= kTmemCols, "S and O fit the tensor memory");
};

struct ChunkInfo {
    float fk, ev, inv_v;  // 2^ek, ev, 2^-ev
    int nv;               // tokens that count
};

// Byte offset of 16-byte piece pc of row r in a swizzled column block.
__device__ __forceinline__ uint32_t swz(int r, int pc) {
    return (uint32_t)(r * 128 + ((pc ^ (r & 7)) << 4));
}

// Sixteen e4m3 bytes -> two 16-byte pieces of fp16.
__device__ __forceinline__ void convert16(const uint4& v, uint4& a, uint4& b) {
    e4m3x4_to_h2(v.x, a.x, a.y);
    e4m3x4_to_h2(v.y, a.z, a.w);
    e4m3x4_to_h2(v.z, b.x, b.y);
    e4m3x4_to_h2(v.w, b.z, b.w);
}

__device__ __forceinline__ uint32_t any_nan(const uint4& v) {
    auto f = [](uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; };
    return f(v.x) | f(v.y) | f(v.z) | f(v.w);
}

// 0x38 (1.0) in every byte that is a NaN, 0 elsewhere.
__device__ __forceinline__ uint32_t nan_ones(uint32_t w) {
    return ((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0x38u;
}
__device__ __forceinline__ uint4 nan_ones(const uint4& v) {
    return make_uint4(nan_ones(v.x), nan_ones(v.y), nan_ones(v.z), nan_ones(v.w));
}
// The bytes with every NaN taken out (0).
__device__ __forceinline__ uint4 without_nan(const uint4& v) {
    auto f = [](uint32_t w) {
        return w & ~(((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu);
    };
    return make_uint4(f(v.x), f(v.y), f(v.z), f(v.w));
}

// A block of the CTA's range: chunks k .. k + cnt - 1 of unit u.
struct Block {
    int u, len, nch;  // the unit, its sequence's tokens, its chunks
    int b, h;         // sequence and KV head of the unit
    int k, cnt;
    bool first, last;  // of its segment
    bool head;         // the segment starts with the unit's first chunk
};

// (sequence, KV head, sub-group) of a unit.
struct Unit {
    int b, h, sg;
    __device__ __forceinline__ Unit(const Kv8DecodeParams& p, int u) {
        b = u / p.units_per_b;
        const int x = u - b * p.units_per_b;
        h = x / p.sub_groups;
        sg = x - h * p.sub_groups;
    }
};

// What a thread's row has come to.
struct RowState {
    float m, mr, l;  // reference, the same less kKv8Lift, this part's sum
    int ev_ref;
    uint32_t ph;     // phase of the barrier that the products arrive at
    bool fail;
};

// Softmax and O += P V of a block, a chunk at a time.  In a function of its own: it
// hardly ever runs, and inside the kernel it takes registers from the path that
// does (64 query tokens of 4 sequences: 56.0 us, against 54.6).  With one block of 16
// tokens in 512 of a 2^20 times larger scale these take 65 us, one in 16: 90.  Every thread
// of the CTA calls it, with S of the block done; on a timeout `fail` is set for all of them.
template <int D>
__device__ __noinline__ void chunks_apart(RowState* st, uint8_t* base, uint32_t lane_base,
                                          uint32_t tmem, float fs, int lim, int cnt, bool fresh) {
    using Lay = Layout<D>;
    float* s_sum = reinterpret_cast<float*>(base + Lay::kOffMax);
    const ChunkInfo* s_chunk = reinterpret_cast<const ChunkInfo*>(base + Lay::kOffChunk);
    const int8_t* s_ev = reinterpret_cast<const int8_t*>(base + Lay::kOffEv);
    uint64_t* bar = reinterpret_cast<uint64_t*>(base + Lay::kOffBar);
    const uint32_t sb = smem_u32(base);
    const int tid = threadIdx.x, row = tid & 127, part = tid >> 7;
    RowState z = *st;
#pragma unroll 1
    for (int c = 0; c < cnt && !z.fail; ++c) {
        const int ev = s_ev[c];
        if (ev == kNoExp) continue;
        const bool low = ev < z.ev_ref - kKv8Span;
        z.ev_ref = low ? ev : max(z.ev_ref, ev);
        s_sum[part * 128 + row] = z.l;
        __syncthreads();
        uint32_t v[16];
        tmem_ld(lane_base + c * kChunk, v);
        const float4 ci = *reinterpret_cast<const float4*>(&s_chunk[c]);
        const int see = min(__float_as_int(ci.w), lim - c * kChunk + 1);
        const float g = fs * ci.x;
        float mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (e < see) mx = fmaxf(mx, __uint_as_float(v[e]));
        if (see > 0) mx = fmaf(mx, g, ci.y);
        float m_new = fmaxf(z.m, mx);
        if (low) {  // down to what suits the row's sum so far
            float l = 0.f;
#pragma unroll
            for (int x = 0; x < kParts; ++x) l += s_sum[x * 128 + row];
            m_new = fminf(m_new, fmaxf(mx, __log2f(l) + z.mr + ci.y));
        }
        float alpha = 1.f;
        if (m_new > -INFINITY) {  // the row has seen a token
            alpha = fast_exp2(z.m - m_new);
            z.m = m_new;
            z.mr = m_new - kKv8Lift;
            z.l *= alpha;
        }
        // 8 of the 16 tokens a thread
        float y[8], sum = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float s = __uint_as_float(part ? v[8 + e] : v[e]);
            y[e] = 8 * part + e < see ? fast_exp2(fmaf(s, g, ci.y - z.mr)) : 0.f;
            sum += y[e];
        }
        z.l = fmaf(sum, ci.z, z.l);
        *reinterpret_cast<uint4*>(base + Lay::kOffK + (c >> 2) * Lay::kColBytes +
                                  swz(row, 2 * (c & 3) + part)) =
            make_uint4(Cvt<__half>::pack2(y[0], y[1]), Cvt<__half>::pack2(y[2], y[3]),
                       Cvt<__half>::pack2(y[4], y[5]), Cvt<__half>::pack2(y[6], y[7]));
        if (!fresh) {
#pragma unroll 1
            for (int x = 0; x < D / kParts; x += 8) {
                const uint32_t at = lane_base + Lay::kColsS + part * (D / kParts) + x;
                uint32_t o[8];
                tmem_ld(at, o);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st(at, o);
            }
            tmem_wait_st();
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
            umma_f16(tmem + Lay::kColsS,
                     umma_sdesc(sb + Lay::kOffK, 16, 1024) +
                         (((c >> 2) * Lay::kColBytes + (c & 3) * 32) >> 4),
                     umma_sdesc(sb + Lay::kOffV, Lay::kColBytes, 1024) + ((c * kChunk * 128) >> 4),
                     umma_idesc(kRows, D, false, true), !fresh);
            umma_commit(bar);
        }
        z.fail = __syncthreads_or(!mbar_wait_bounded(bar, z.ph));
        if (!z.fail) z.ph ^= 1u;
        tc_fence_after();
        fresh = false;
    }
    *st = z;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 2)
kv8_umma_kernel(const __grid_constant__ Kv8DecodeParams p, const uint8_t* k_pool,
                const uint8_t* v_pool) {
    using Lay = Layout<D>;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    constexpr int PPR = D / 16;    // 16-byte pieces of a token's e4m3 row
    constexpr int RPP = 32 / PPR, LOADS = kChunk / RPP;  // token rows of a warp's pass; passes
    static_assert(kThreads / 32 == kBlockChunks, "a warp a chunk");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
    uint8_t* base = smem_raw + pad;
    const uint32_t sb = raw + pad;
    float* s_max = reinterpret_cast<float*>(base + Lay::kOffMax);
    ChunkInfo* s_chunk = reinterpret_cast<ChunkInfo*>(base + Lay::kOffChunk);
    int8_t* s_ev = reinterpret_cast<int8_t*>(base + Lay::kOffEv);
    uint64_t* bar = reinterpret_cast<uint64_t*>(base + Lay::kOffBar);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar + 1);
    uint32_t* s_flags = tmem_slot + 1;
    int32_t* s_prefix = reinterpret_cast<int32_t*>(base + Lay::kOffPlan);
    const int tid = threadIdx.x, warp = tid >> 5;
    const int row = tid & 127, part = tid >> 7;

    if (warp == 0) tmem_alloc(tmem_slot, Lay::kTmemCols);
    if (tid == 32) {
        mbar_init(bar, 1);
        *s_flags = 0;
        fence_barrier_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t lane_base = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const bool early = p.after_append && p.self_plan;  // as in kv8_decode.cuh
    if (!early) pdl_wait();

    uint32_t flags = 0;
    const int32_t* prefix;
    int nw, sw, rr;
    if (p.self_plan) {
        const int total = kv8_self_plan<kThreads>(p, s_prefix, &flags);
        prefix = s_prefix;
        kv8_ranges(total, p.workers_req, p.workers_auto, &nw, &sw, &rr);
        if (blockIdx.x == 0 && tid == 0) {
            p.hdr->num_workers = nw;
            p.hdr->chunks_per_worker = sw;
            p.hdr->extra_chunks = rr;
        }
    } else {
        prefix = p.prefix;
        nw = p.hdr->num_workers;
        sw = p.hdr->chunks_per_worker;
        rr = p.hdr->extra_chunks;
    }
    if (early) pdl_wait();
    const int cta = blockIdx.x;
    const int f0 = range_begin(cta, sw, rr);
    const int f_end = cta < nw ? f0 + sw + (cta < rr ? 1 : 0) : f0;
    // rows of sequences with no tokens are zeros
    for (int b = cta; b < p.batch; b += gridDim.x) {
        if (prefix[b] != prefix[b + 1] && nw > 0) continue;
        const long long vecs = (long long)p.rows.n_queries * p.rows.n_q_heads * D / 8;
        uint4* dst = reinterpret_cast<uint4*>(p.out) + b * vecs;
        for (long long x = tid; x < vecs; x += kThreads) dst[x] = make_uint4(0u, 0u, 0u, 0u);
    }

    // The next block from position f on; false at the range's end.  (Every thread
    // does the same.)
    int f = f0;
    Block nx;
    nx.u = -1;
    nx.k = nx.cnt = nx.nch = 0;
    auto advance = [&]() -> bool {
        if (nx.u >= 0 && !nx.last) {
            nx.k += nx.cnt;
            nx.first = false;
        } else {
            while (true) {
                if (f >= f_end) return false;
                int lo = 0, hi = p.batch;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (prefix[mid] <= f) lo = mid; else hi = mid;
                }
                const int first = prefix[lo];
                const int per_unit = (prefix[lo + 1] - first) / p.units_per_b;
                const int uidx = (f - first) / per_unit;
                const int k = f - first - uidx * per_unit - p.unit_cost;
                if (k < 0) {  // the unit's cost positions hold nothing
                    f -= k;
                    continue;
                }
                nx.u = lo * p.units_per_b + uidx;
                nx.b = lo;
                nx.h = uidx / p.sub_groups;
                nx.len = (int)min((long long)p.lens[lo], p.cap);
                nx.nch = per_unit - p.unit_cost;
                nx.k = k;
                nx.first = true;
                nx.head = k == 0;
                break;
            }
        }
        nx.cnt = min(kBlockChunks, min(nx.nch - nx.k, f_end - f));
        f += nx.cnt;
        nx.last = nx.k + nx.cnt == nx.nch || f >= f_end;
        return true;
    };

    // A warp brings one chunk of a block: lane (rr, pc) the pieces pc of token rows
    // rr + RPP i, K's and V's at different times (the L1 that the shared memory
    // leaves holds the lines of about one side of two CTAs on the way; more loads
    // wait for room), past L1, which has no use for them (16 query tokens of 32
    // sequences: 83.6 us, through L1 84.4).  The page id of its chunk of the block
    // after is asked for at
    // the same time, so that no load waits for another one inside a segment.
    const int lane = tid & 31, pc = lane % PPR, rr0 = lane / PPR;
    uint4 kr[LOADS], vr[LOADS];
    int page_after = -1;  // page of this warp's chunk of the block after the next one
    int nv = 0;           // tokens of its chunk of the next block that count (bad pages: 0)
    uint32_t sc = 0u;     // the chunk's scale bytes
    long long at = 0;     // this lane's first piece of it
    auto page_of = [&](const Block& c, int k) {
        return __ldg(p.table + (long long)c.b * p.table_stride + kv8_page_col(k, p.page_magic));
    };
    auto load_side = [&](const uint8_t* pool, uint4 (&v)[LOADS]) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            v[i] = make_uint4(0u, 0u, 0u, 0u);  // rows behind the sequence's end
            if (rr0 + RPP * i < nv)
                v[i] = __ldcg(reinterpret_cast<const uint4*>(pool + at + i * (RPP * D)));
        }
    };
    auto fetch_k = [&](const Block& c) {
        const int k = c.k + warp;
        int page = page_after;
        if (c.first && warp < c.cnt) page = page_of(c, k);
        nv = 0;
        sc = 0u;
        if (warp < c.cnt) {
            if (page >= 0 && page < p.num_pages) {
                nv = min(kChunk, c.len - k * kChunk);
                const long long blk =
                    (long long)(page * p.n_kv_heads + c.h) * p.chunks_per_page +
                    (k - kv8_page_col(k, p.page_magic) * p.chunks_per_page);
                at = blk * (kChunk * D) + rr0 * D + pc * 16;
                sc = (uint32_t)p.scales[blk];
            } else {
                flags |= PKV_DEV_BAD_PAGE;
            }
        }
        load_side(k_pool, kr);
        if (!c.last && k + c.cnt < c.nch) page_after = page_of(c, k + c.cnt);
    };
    auto fetch_v = [&]() { load_side(v_pool, vr); };
    // 16 converted bytes into the tile at `off`: pieces 2 q, 2 q + 1 of a row (the
    // upper column block's in the other order, so that a row's stores hit
    // different banks)
    auto put = [&](int off, int r, const uint4& v) {
        uint4 a, b;
        convert16(v, a, b);
        const int blk = pc >> 2, q = (pc & 3) * 2;
        uint8_t* t = base + off + blk * Lay::kColBytes;
        const int o = blk & 1;
        *reinterpret_cast<uint4*>(t + swz(r, q + o)) = o ? b : a;
        *reinterpret_cast<uint4*>(t + swz(r, q + 1 - o)) = o ? a : b;
    };

    uint32_t ph = 0;
    bool fail = false;  // a wait gave up: the same for the whole CTA
    float m_run = -INFINITY, mr = 0.f, l_run = 0.f, fs = 0.f;
    int ev_ref = kNoExp;           // the V exponent that m suits (kv8.cuh)
    int lim_row = 0, lim_min = 0;  // last token that this thread's row, the unit's first row, sees
    // Wait for the products in flight; true: given up.  Every thread learns the same, so
    // nobody touches what products may still use after anybody gave up.
    auto wait_all = [&]() -> bool {
        const bool late = __syncthreads_or(!mbar_wait_bounded(bar, ph));
        if (!late) ph ^= 1u;
        tc_fence_after();
        return late;
    };
    Block cur;
    bool more = advance();
    if (more) {
        fetch_k(nx);
        fetch_v();
    }
    while (more) {
        cur = nx;
        if (cur.first) {
            const Unit un(p, cur.u);
            // ---- the unit's queries to fp16 (bf16: times a power of two that puts
            // the row's largest element into [2^14, 2^15); a negative scale's sign
            // goes into them, so that the factors below are positive): D / 8 lanes
            // a row, a 16-byte vector each
            constexpr int LPR = D / 8, RPW = 32 / LPR;  // lanes a row; rows of a warp side by side
            constexpr int PASSES = kRows / (kThreads / 32) / RPW;
            const int qp = lane % LPR;
            const int rows = p.rows.rows(un.sg);
            uint4 q[PASSES];
#pragma unroll
            for (int x = 0; x < PASSES; ++x) {
                const int r = (warp * PASSES + x) * RPW + lane / LPR;
                q[x] = make_uint4(0u, 0u, 0u, 0u);
                if (r < rows)
                    q[x] = reinterpret_cast<const uint4*>(
                        static_cast<const T*>(p.q) + p.rows.row(un.b, un.h, un.sg, r) * D)[qp];
            }
#pragma unroll
            for (int x = 0; x < PASSES; ++x) {
                const int r = (warp * PASSES + x) * RPW + lane / LPR;
                int shift = 0;
                if constexpr (kBf16) {
                    uint32_t mx = __vmaxu2(__vmaxu2(q[x].x & 0x7fff7fffu, q[x].y & 0x7fff7fffu),
                                           __vmaxu2(q[x].z & 0x7fff7fffu, q[x].w & 0x7fff7fffu));
                    mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
                    for (int o = LPR / 2; o > 0; o >>= 1)
                        mx = max(mx, __shfl_xor_sync(kFull, mx, o));
                    shift = mx == 0u ? 0 : min(141 - (int)(mx >> 7), 126);
                }
                const float g = p.scale_log2 < 0.f ? -exp2i(shift) : exp2i(shift);
                auto cv = [&](uint32_t w) {
                    if constexpr (kBf16)
                        return Cvt<__half>::pack2(__uint_as_float(w << 16) * g,
                                                  __uint_as_float(w & 0xffff0000u) * g);
                    else
                        return p.scale_log2 < 0.f ? w ^ 0x80008000u : w;
                };
                *reinterpret_cast<uint4*>(base + Lay::kOffQ + (qp >> 3) * Lay::kColBytes +
                                          swz(r, qp & 7)) =
                    make_uint4(cv(q[x].x), cv(q[x].y), cv(q[x].z), cv(q[x].w));
                if (qp == 0) s_max[r] = fabsf(p.scale_log2) * exp2i(-shift);
            }
            __syncthreads();
            fs = s_max[row];
            m_run = -INFINITY;
            mr = 0.f;
            l_run = 0.f;
            ev_ref = kNoExp;
            const int last = cur.len - p.rows.n_queries;
            lim_min = last + p.rows.first_query(un.sg);
            lim_row = min(last + p.rows.query(un.sg, row), cur.len - 1);
        }
        const int ntok = cur.cnt * kChunk, tok0 = cur.k * kChunk;
        const bool masked = cur.len - tok0 < ntok || tok0 + ntok - 1 > lim_min;
        const int lim = lim_row - tok0;

        // ---- S = Q K^T of the converted K
#pragma unroll
        for (int i = 0; i < LOADS; ++i) put(Lay::kOffK, warp * kChunk + rr0 + RPP * i, kr[i]);
        const int e = kv8_clamp_exp((int)(sc >> 8) - 127), ev = nv > 0 ? e : kNoExp;
        if (lane == 0) {
            s_chunk[warp] = {__uint_as_float((sc & 0xffu) << 23), (float)e, exp2i(-e), nv};
            s_ev[warp] = (int8_t)ev;
        }
        fence_proxy_async_smem();
        tc_fence_before();
        // an exponent out of the band that m suits?
        const bool look =
            __syncthreads_or(ev != kNoExp && (ev > ev_ref || ev < ev_ref - kKv8Span));
        if (tid == 0) {
            tc_fence_after();
            const uint32_t idesc = umma_idesc(kRows, ntok, false, false);
            const uint64_t qd = umma_sdesc(sb + Lay::kOffQ, 16, 1024);
            const uint64_t kd = umma_sdesc(sb + Lay::kOffK, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * Lay::kColBytes + (kk & 3) * 32) >> 4;
                umma_f16(tmem, qd + off, kd + off, idesc, kk > 0);
            }
            umma_commit(bar);
        }
        // ---- beside it: V converted (its place is free, the product before is done)
        uint32_t nan = 0u;
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            uint4 v = vr[i];
            if (masked) {
                nan |= any_nan(v);
                v = without_nan(v);
            }
            put(Lay::kOffV, warp * kChunk + rr0 + RPP * i, v);
        }
        more = advance();
        if (more) fetch_k(nx);  // comes behind the product and the softmax
        fail = wait_all();
        if (fail) break;
        // D (+)= P V
        auto product = [&](uint32_t d, bool keep) {
            tc_fence_after();
            const uint32_t idesc = umma_idesc(kRows, D, false, true);
            const uint64_t pd = umma_sdesc(sb + Lay::kOffK, 16, 1024);
            const uint64_t vd = umma_sdesc(sb + Lay::kOffV, Lay::kColBytes, 1024);
#pragma unroll
            for (int kt = 0; kt < kBlockChunks; ++kt)
                if (kt < cur.cnt)
                    umma_f16(d, pd + (((kt >> 2) * Lay::kColBytes + (kt & 3) * 32) >> 4),
                             vd + ((kt * kChunk * 128) >> 4), idesc, keep || kt > 0);
            umma_commit(bar);
        };
        bool apart = false;  // too far from each other, or all below ev_ref's band
        if (look) {
            int hi = ev_ref, lo = kKv8MaxExp;
#pragma unroll
            for (int c = 0; c < kBlockChunks; ++c) {
                const int x = s_ev[c];
                hi = max(hi, x);
                if (c < cur.cnt && x != kNoExp) lo = min(lo, x);
            }
            apart = lo < hi - kKv8Span;
            if (!apart) ev_ref = hi;
        }
        bool fix = false;
        if (__builtin_expect(apart, 0)) {
            fix = masked && __syncthreads_or(nan != 0u);
            RowState z = {m_run, mr, l_run, ev_ref, ph, false};
            chunks_apart<D>(&z, base, lane_base, tmem, fs, lim, cur.cnt, cur.first);
            m_run = z.m;
            mr = z.mr;
            l_run = z.l;
            ev_ref = z.ev_ref;
            ph = z.ph;
            fail = z.fail;
            if (fail) break;
            if (more && !fix) fetch_v();
        } else {
            // ---- softmax: this thread's part of row `row`
            // (twice out of tensor memory, for the maximum and for the weights, a chunk at
            // a time: beside the next block's bytes there are no registers for more, and
            // what the compiler moves to local memory instead does not stay in the little
            // L1 that the shared memory leaves)
            float mx = -INFINITY;
            const bool have = part * kPartChunks < cur.cnt;
            if (have) {
#pragma unroll
                for (int c = 0; c < kPartChunks; ++c) {
                    const int ch = part * kPartChunks + c;
                    if (ch >= cur.cnt) break;
                    uint32_t v[16];
                    tmem_ld(lane_base + ch * kChunk, v);
                    const float4 ci = *reinterpret_cast<const float4*>(&s_chunk[ch]);
                    // tokens of the chunk that the row sees (bad pages: none)
                    const int see = min(__float_as_int(ci.w), lim - ch * kChunk + 1);
                    float top = -INFINITY;
                    if (see >= kChunk) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) top = fmaxf(top, __uint_as_float(v[e]));
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (e < see) top = fmaxf(top, __uint_as_float(v[e]));
                    }
                    if (see > 0) mx = fmaxf(mx, fmaf(top, fs * ci.x, ci.y));
                }
            }
            s_max[part * 128 + row] = mx;
            // the warps that share these 32 rows
            asm volatile("bar.sync %0, %1;" ::"r"(1 + (warp & 3)), "n"(kParts * 32) : "memory");
#pragma unroll
            for (int x = 0; x < kParts; ++x) mx = fmaxf(mx, s_max[x * 128 + row]);
            float alpha = 1.f;
            if (mx > m_run + kKv8Slack) {
                mr = mx - kKv8Lift;  // finite, or +inf (then NaN, as it should be)
                alpha = fast_exp2(m_run - mx);
                m_run = mx;
                l_run *= alpha;
            }
            // the products S = Q K^T of the block are done: K's place takes P
            if (have) {
#pragma unroll
                for (int c = 0; c < kPartChunks; ++c) {
                    const int ch = part * kPartChunks + c;
                    if (ch >= cur.cnt) break;
                    uint32_t v[16];
                    float y[16];
                    tmem_ld(lane_base + ch * kChunk, v);
                    const float4 ci = *reinterpret_cast<const float4*>(&s_chunk[ch]);
                    const int see = min(__float_as_int(ci.w), lim - ch * kChunk + 1);
                    const float g = fs * ci.x, off = ci.y - mr;
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        y[e] = fast_exp2(fmaf(__uint_as_float(v[e]), g, off));
                    if (see < kChunk) {
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (e >= see) y[e] = 0.f;
                    }
                    float sum = 0.f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum += y[e];
                    l_run = fmaf(sum, ci.z, l_run);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float* w = y + 8 * q;
                        *reinterpret_cast<uint4*>(base + Lay::kOffK + (ch >> 2) * Lay::kColBytes +
                                                  swz(row, 2 * (ch & 3) + q)) =
                            make_uint4(
                                Cvt<__half>::pack2(w[0], w[1]), Cvt<__half>::pack2(w[2], w[3]),
                                Cvt<__half>::pack2(w[4], w[5]), Cvt<__half>::pack2(w[6], w[7]));
                    }
                }
            }
            // the earlier blocks' O to the new reference: its part of the columns a thread
            if (!cur.first && __any_sync(kFull, alpha != 1.f)) {
#pragma unroll
                for (int x = 0; x < D / kParts; x += 16) {
                    const uint32_t at = lane_base + Lay::kColsS + part * (D / kParts) + x;
                    uint32_t v[16];
                    tmem_ld(at, v);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        v[e] = __float_as_uint(__uint_as_float(v[e]) * alpha);
                    tmem_st(at, v);
                }
                tmem_wait_st();
            }
            fence_proxy_async_smem();
            tc_fence_before();
            // A NaN in V at a token that some row does not see must not reach that row
            // through its weight 0: such a block is multiplied without its NaNs, and
            // below they are given back to the rows that see them.
            fix = __syncthreads_or(nan != 0u);  // (looked for in masked blocks only)
            if (more && !fix) fetch_v();
            // ---- O += P V
            if (tid == 0) product(tmem + Lay::kColsS, !cur.first);
            fail = wait_all();
            if (fail) break;
        }
        if (fix) {
            // which outputs see a NaN: (row sees token) x (NaN at token), counted
            // in S's place
#pragma unroll
            for (int i = 0; i < LOADS; ++i) put(Lay::kOffV, warp * kChunk + rr0 + RPP * i, nan_ones(vr[i]));
#pragma unroll
            for (int q = 0; q < 2 * kPartChunks; ++q) {
                uint32_t w[4];
                const int piece = part * 2 * kPartChunks + q;  // 8 tokens
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int t = 8 * piece + 2 * e;
                    w[e] = (t <= lim ? 0x3c00u : 0u) | (t + 1 <= lim ? 0x3c000000u : 0u);
                }
                *reinterpret_cast<uint4*>(base + Lay::kOffK + (piece >> 3) * Lay::kColBytes +
                                          swz(row, piece & 7)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncthreads();
            if (tid == 0) product(tmem, false);
            fail = wait_all();
            if (fail) break;
#pragma unroll 1
            for (int x = 0; x < D / kParts; x += 8) {
                uint32_t n[8], v[8];
                tmem_ld(lane_base + part * (D / kParts) + x, n);
                tmem_ld(lane_base + Lay::kColsS + part * (D / kParts) + x, v);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (__uint_as_float(n[e]) > 0.f) v[e] = 0x7fc00000u;
                tmem_st(lane_base + Lay::kColsS + part * (D / kParts) + x, v);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncthreads();
            if (more) fetch_v();
        }

        // ---- the segment's end
        if (cur.last) {
            s_max[part * 128 + row] = l_run;
            __syncthreads();
            float l = 0.f;
#pragma unroll
            for (int x = 0; x < kParts; ++x) l += s_max[x * 128 + row];
            const Unit un(p, cur.u);
            const int rows = p.rows.rows(un.sg);
            const bool whole = cur.head && cur.k + cur.cnt == cur.nch;
            const float inv = l == 0.f ? 0.f : 1.0f / l;  // no token seen: zeros
            float* slot = p.partials + (long long)(cur.u + cta) * partial_slot_floats(p.gs, D);
#pragma unroll
            for (int x = 0; x < D / kParts; x += 16) {
                const int c0 = part * (D / kParts) + x;
                uint32_t v[16];
                tmem_ld(lane_base + Lay::kColsS + c0, v);
                if (row < rows) {
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(
                            static_cast<T*>(p.out) +
                            p.rows.row(un.b, un.h, un.sg, row) * D + c0);
                        auto pk = [&](int e) {
                            return Cvt<T>::pack2(__uint_as_float(v[e]) * inv,
                                                 __uint_as_float(v[e + 1]) * inv);
                        };
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            dst[e] = make_uint4(pk(8 * e), pk(8 * e + 2), pk(8 * e + 4),
                                                pk(8 * e + 6));
                    } else {
                        uint4* dst = reinterpret_cast<uint4*>(slot + (long long)row * D + c0);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            dst[e] = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2],
                                                v[4 * e + 3]);
                    }
                }
            }
            if (!whole && row < rows && part == 0) {
                slot[p.gs * D + row] = m_run;
                slot[p.gs * D + p.gs + row] = l;
            }
            tc_fence_before();  // O is read before the next unit's first product
            __syncthreads();
        }
    }
    if (fail) {
        flags |= PKV_DEV_TIMEOUT;
        mbar_wait_bounded(bar, ph);  // once more for the products in flight
    }
    if (flags) atomicOr(s_flags, flags);
    tc_fence_before();
    __syncthreads();
    if (tid == 0) p.flags[cta] = *s_flags;
    pdl_trigger();
    if (warp == 0) tmem_dealloc(tmem, Lay::kTmemCols);
}

template <typename T, int D>
Kv8DecodeInfo info() {
    Kv8DecodeInfo i;
    i.umma = kv8_umma_kernel<T, D>;
    i.warps = 1;  // a worker is a CTA
    i.threads = kThreads;
    i.smem_bytes = Layout<D>::kBytes;
    return i;
}

}  // namespace

Kv8DecodeInfo kv8_umma_info(bool bf16, int head_dim) {
    if (bf16) return head_dim == 128 ? info<__nv_bfloat16, 128>() : info<__nv_bfloat16, 64>();
    return head_dim == 128 ? info<__half, 128>() : info<__half, 64>();
}

}  // namespace pkv
