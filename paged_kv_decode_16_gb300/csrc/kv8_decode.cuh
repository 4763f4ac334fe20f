// kv8_decode.cuh -- decode attention over the 8-bit paged cache.
//
// Work split, chunk pipeline and partial states are those of the 16-bit kernel
// (schedule.cuh, decode_mma.cuh): a warp per balanced range of 16-token
// chunks, a ring of chunk buffers per warp filled by tensor copies, fp32
// partial states merged by the combine kernel.  A chunk is exactly one block of
// the cache, so it has one K scale 2^ek and one V scale 2^ev.
//
// Mathematics.  With x_t = (scale * log2 e) q.k8_t 2^ek(t) + ev(t), a running
// reference m and p_t = 2^(x_t - m):
//     o += p_t v8_t,   l += p_t 2^-ev(t),   out = o / l,
// since p_t v8_t = 2^(s_t - m) (v8_t 2^ev).  The V scale thus costs one add in
// the exponent, the largest p is about 1 whatever the scales are, and (m, l, o)
// merge like any other partial states.  (A term of l weighs 2^(s_t - m); a
// block whose p has left fp32's range, below 2^-126, still has no weight in l
// because the scales span at most 2^100.)
//
// Both products run transposed on m16n8k16 (fp16 in, fp32 accumulate), the 16
// tokens (S^T = K Q^T) or 16 elements of a head (O^T = V^T P^T) as the rows and
// 8 query rows as the columns: a GQA group of 4 to 8 fills a tile that would
// be half empty the other way round.  e4m3 is exact in fp16, so the cache
// enters without rounding.  bf16 queries are scaled by a power of two per row
// (largest element in [2^14, 2^15)) and are exact in fp16 down to 2^-31 of the
// row's largest element.  P is rounded to fp16 (11 bits, relative error at most
// 2^-11 a weight), as in the 16-bit kernel.
//
// The order of k in a product is free as long as both operands agree.  For
// S^T lane (j = lane / 4, t = lane % 4) takes D/4 consecutive elements of token
// j's row, for O^T D/8 consecutive elements of tokens 2t, 2t+1, 2t+8 and 2t+9:
// 16-byte shared loads straight from the copied rows, no transposing loads;
// with the copies' swizzle they hit every bank once (D = 64: V's twice).
#pragma once

#include <cuda.h>

#include <type_traits>

#include "decode_mma.cuh"
#include "kv8.cuh"
#include "merge.cuh"
#include "schedule.cuh"

namespace pkv {

// The scales of a lane's chunk.
struct Kv8Extra {
    const uint16_t* scales;
    uint32_t v;  // bytes: K, V
    __device__ __forceinline__ void load(const ChunkDesc& d) {
        v = d.off >= 0 ? (uint32_t)__ldg(scales + (d.off >> 4)) : 0u;
    }
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

// Shared memory of one CTA: every warp's ring of K/V stages, then (units of
// more than 16 rows) every warp's query fragments, then the mbarriers.
template <int D, int NT, int STAGES, int WARPS>
struct Kv8Layout {
    static constexpr int kSide = kChunk * D;            // K or V bytes of a chunk
    static constexpr int kStageBytes = 2 * kSide;
    static constexpr int kWarpKV = STAGES * kStageBytes;
    static constexpr bool kQShared = NT > 2;
    static constexpr int kWarpQ = kQShared ? NT * 8 * D * 2 : 0;
    static constexpr int kOffQ = WARPS * kWarpKV;
    static constexpr int kOffBar = kOffQ + WARPS * kWarpQ;
    static constexpr int kBytes = kOffBar + WARPS * STAGES * 8 + 1024;  // + alignment slack
};

// NT tiles of 8 query rows; a unit has at most 8 NT rows.
template <typename T, int D, int NT, int WARPS, int STAGES>
__global__ void __launch_bounds__(WARPS * 32)
kv8_decode_kernel(const Kv8DecodeParams kp, const __grid_constant__ CUtensorMap kmap,
                  const __grid_constant__ CUtensorMap vmap) {
    using Lay = Kv8Layout<D, NT, STAGES, WARPS>;
    constexpr int KSTEPS = D / 16;  // k-steps of S^T
    constexpr int MT = D / 16;      // m16 tiles of O^T
    constexpr int DPL = D / 8;      // V elements a lane takes of a row
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    // a row's scores may pass m by this much (in binary orders) before m moves:
    // p stays below 2^8, far inside fp16, and after a range's first chunk the
    // accumulators are hardly ever rescaled
    constexpr float kSlack = 8.f;
    const DecodeParams& p = kp.d;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;  // the swizzle's period
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    uint8_t* base = smem_raw + pad;
    uint8_t* wsm = base + warp * Lay::kWarpKV;
    const uint32_t wsm_u32 = raw + pad + warp * Lay::kWarpKV;
    // query fragments in shared memory: 16-byte vector x of tile n at
    // (n * KSTEPS / 2 + x) * 512 + lane * 16
    const uint32_t sq = raw + pad + Lay::kOffQ + warp * Lay::kWarpQ + lane * 16;
    uint64_t* bar = reinterpret_cast<uint64_t*>(base + Lay::kOffBar) + warp * STAGES;

    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < STAGES; ++s) mbar_init(&bar[s], 1);
        fence_barrier_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap))
                     : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap))
                     : "memory");
    }
    __syncwarp();
    pdl_wait();

    const int nw = p.hdr->num_workers;
    const int gw = blockIdx.x * WARPS + warp;
    const int all_warps = gridDim.x * WARPS;
    if (gw >= nw) {
        zero_empty_sequences(p, D, gw, all_warps, lane);
        return;
    }
    WorkStreamT<Kv8Extra> ws;
    ws.xa.scales = ws.xb.scales = kp.scales;
    ws.xa.v = ws.xb.v = 0u;
    ws.init(p, lane, gw);
    if (ws.stream_end == 0) {
        zero_empty_sequences(p, D, gw, all_warps, lane);
        return;
    }

    const int units_per_b = ws.units_per_b;
    const uint64_t kv_policy = l2_evict_first_policy();
    const int j = lane >> 2, t = lane & 3;

    // Issue the copies of stream position i into stage i % STAGES; false past
    // the end of the stream.
    auto issue = [&](int i) -> bool {
        if (!ws.covered(p, i)) return false;
        const bool second = i >= ws.a_end();
        const int src = i - (second ? ws.b_start : ws.a_start);
        const long long off = __shfl_sync(kFull, second ? ws.wb.off : ws.wa.off, src);
        if (lane == 0) {
            const int st = i % STAGES;
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(&bar[st], off >= 0 ? (uint32_t)Lay::kStageBytes : 0u);
            if (off >= 0) {
                uint8_t* stage = wsm + st * Lay::kStageBytes;
                tma_load_2d_hint(stage, &kmap, 0, (int)off, &bar[st], kv_policy);
                tma_load_2d_hint(stage + Lay::kSide, &vmap, 0, (int)off, &bar[st], kv_policy);
            }
        }
        return true;
    };

    int issued = 0;
    while (issued < STAGES && issue(issued)) ++issued;
    zero_empty_sequences(p, D, gw, all_warps, lane);  // while the first copies are in flight

    uint32_t qf[Lay::kQShared ? 1 : NT][KSTEPS][2];  // B fragments of Q^T
    float fs[NT][2];   // score factors of rows 2t, 2t+1 of a tile: scale log2(e) / row scale
    float o[NT][MT][4];  // O^T: elements DPL j + 2i (c0, c1) and + 1 (c2, c3) of rows 2t, 2t+1
    float m[NT][2], mr[NT][2];  // reference of rows 2t, 2t+1; the same with 0 for -inf
    float l[NT][2];             // this lane's part of the rows' sums
    int lim[NT][2];             // last token that rows 2t, 2t+1 see
    int lim_min = 0;            // the smallest of the unit's
    int seg_rows = 0, seg_slot = 0;
    bool seg_whole_start = false;

    auto give_up = [&](int from) {
        if (lane == 0) set_status(p.status, PKV_DEV_TIMEOUT);
        for (int i = from; i < issued; ++i)
            mbar_wait_bounded(&bar[i % STAGES], (uint32_t)((i / STAGES) & 1));
    };

    for (int i = 0; i < ws.stream_end; ++i) {
        ws.consumer_at(p, i, STAGES + 1);
        const ChunkDesc d = ws.fetch(i);
        const bool in_b = i >= ws.a_end();
        const uint32_t sc = __shfl_sync(kFull, in_b ? ws.xb.v : ws.xa.v,
                                        i - (in_b ? ws.b_start : ws.a_start));
        const int st = i % STAGES;
        if (ws.seg_start(i, d)) {
            const int b = d.u / units_per_b;
            const int uidx = d.u - b * units_per_b;
            const int h = uidx / p.sub_groups;
            const int sg = uidx - h * p.sub_groups;
            seg_rows = p.rows.rows(sg);
            seg_slot = ws.slot_base + d.u;
            seg_whole_start = d.k == 0;
            const int last = d.len - p.rows.n_queries;
            lim_min = last + p.rows.first_query(sg);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                // lane (j, t) takes elements D/4 t .. of row 8n + j
                uint32_t u[KSTEPS * 2];
                const int r = 8 * n + j;
                const bool ok = r < seg_rows;
                const uint4* src = reinterpret_cast<const uint4*>(
                    static_cast<const T*>(p.q) + (ok ? p.rows.row(b, h, sg, r) * D : 0) + t * (D / 4));
#pragma unroll
                for (int x = 0; x < KSTEPS / 2; ++x) {
                    const uint4 v = ok ? src[x] : make_uint4(0u, 0u, 0u, 0u);
                    u[4 * x] = v.x;
                    u[4 * x + 1] = v.y;
                    u[4 * x + 2] = v.z;
                    u[4 * x + 3] = v.w;
                }
                int shift = 0;  // the row is multiplied by 2^shift
                if constexpr (kBf16) {
                    uint32_t mx = 0u;
#pragma unroll
                    for (int x = 0; x < KSTEPS * 2; ++x) mx = __vmaxu2(mx, u[x] & 0x7fff7fffu);
                    mx = max(mx & 0xffffu, mx >> 16);
                    mx = max(mx, __shfl_xor_sync(kFull, mx, 1));
                    mx = max(mx, __shfl_xor_sync(kFull, mx, 2));
                    shift = mx == 0u ? 0 : min(141 - (int)(mx >> 7), 126);
                    const float f = exp2i(shift);
#pragma unroll
                    for (int x = 0; x < KSTEPS * 2; ++x)
                        u[x] = Cvt<__half>::pack2(__uint_as_float(u[x] << 16) * f,
                                                  __uint_as_float(u[x] & 0xffff0000u) * f);
                }
                if constexpr (Lay::kQShared) {
#pragma unroll
                    for (int x = 0; x < KSTEPS / 2; ++x)
                        sts128(sq + (n * (KSTEPS / 2) + x) * 512,
                               make_uint4(u[4 * x], u[4 * x + 1], u[4 * x + 2], u[4 * x + 3]));
                } else {
#pragma unroll
                    for (int kk = 0; kk < KSTEPS; ++kk) {
                        qf[n][kk][0] = u[2 * kk];
                        qf[n][kk][1] = u[2 * kk + 1];
                    }
                }
                // factors and limits of the rows this lane's accumulators hold
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int sh = __shfl_sync(kFull, shift, 4 * (2 * t + c));
                    fs[n][c] = p.scale_log2 * exp2i(-sh);
                    lim[n][c] = last + p.rows.query(sg, 8 * n + 2 * t + c);
                    m[n][c] = -INFINITY;
                    mr[n][c] = 0.f;
                    l[n][c] = 0.f;
                }
#pragma unroll
                for (int x = 0; x < MT; ++x) o[n][x][0] = o[n][x][1] = o[n][x][2] = o[n][x][3] = 0.f;
            }
        }
        if (!mbar_wait_bounded(&bar[st], (uint32_t)((i / STAGES) & 1))) {
            give_up(i + 1);
            return;
        }

        if (d.off >= 0) {
            const uint32_t kst = wsm_u32 + st * Lay::kStageBytes;
            const uint32_t vst = kst + Lay::kSide;
            const int tok0 = d.k * kChunk;
            const float fk = __uint_as_float((sc & 0xffu) << 23);  // 2^ek (byte 0: 0)
            const int evi = kv8_clamp_exp((int)(sc >> 8) - 127);
            const float ev = (float)evi, inv_v = exp2i(-evi);
            // ---- S^T = K Q^T ----
            uint32_t kw[2][KSTEPS];  // rows j and j + 8: D/4 bytes each
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                const int row = j + 8 * hf;
                if constexpr (D == 128) {
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint4 v = lds128(kst + row * 128 + (((2 * t + x) ^ (row & 7)) << 4));
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
            float s[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
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
                        mma_f16(s[n], a[0][0], a[0][1], a[0][2], a[0][3], q4.x, q4.y);
                        mma_f16(s[n], a[1][0], a[1][1], a[1][2], a[1][3], q4.z, q4.w);
                    } else {
                        mma_f16(s[n], a[0][0], a[0][1], a[0][2], a[0][3], qf[n][kk][0],
                                qf[n][kk][1]);
                        mma_f16(s[n], a[1][0], a[1][1], a[1][2], a[1][3], qf[n][kk + 1][0],
                                qf[n][kk + 1][1]);
                    }
                }
            }
            // ---- exponents; masks only where the chunk passes a row's last token ----
            const bool masked = tok0 + kChunk - 1 > min(lim_min, d.len - 1);
            bool above = false;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float f0 = fs[n][0] * fk, f1 = fs[n][1] * fk;
                s[n][0] = fmaf(s[n][0], f0, ev);
                s[n][1] = fmaf(s[n][1], f1, ev);
                s[n][2] = fmaf(s[n][2], f0, ev);
                s[n][3] = fmaf(s[n][3], f1, ev);
                if (masked) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int tok = j + 8 * (c >> 1);
                        if (tok >= d.nvalid || tok0 + tok > lim[n][c & 1]) s[n][c] = -INFINITY;
                    }
                }
                above |= fmaxf(s[n][0], s[n][2]) > m[n][0] + kSlack ||
                         fmaxf(s[n][1], s[n][3]) > m[n][1] + kSlack;
            }
            if (__any_sync(kFull, above)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float mx = fmaxf(s[n][c], s[n][c + 2]);
                        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
                        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
                        mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
                        const float m_new = fmaxf(m[n][c], mx);
                        // a row that has seen no token yet: reference 0, weights 0
                        mr[n][c] = m_new == -INFINITY ? 0.f : m_new;
                        const float alpha = fast_exp2(m[n][c] - mr[n][c]);
                        m[n][c] = m_new;
                        l[n][c] *= alpha;
#pragma unroll
                        for (int x = 0; x < MT; ++x) {
                            o[n][x][c] *= alpha;
                            o[n][x][c + 2] *= alpha;
                        }
                    }
            }
            uint32_t pb[NT][2];  // B fragments of P^T: tokens 2t, 2t+1 (+ 8) of row j
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float p0 = fast_exp2(s[n][0] - mr[n][0]), p1 = fast_exp2(s[n][1] - mr[n][1]);
                const float p2 = fast_exp2(s[n][2] - mr[n][0]), p3 = fast_exp2(s[n][3] - mr[n][1]);
                l[n][0] = fmaf(p0 + p2, inv_v, l[n][0]);
                l[n][1] = fmaf(p1 + p3, inv_v, l[n][1]);
                pb[n][0] = transpose8x8(Cvt<__half>::pack2(p0, p1));
                pb[n][1] = transpose8x8(Cvt<__half>::pack2(p2, p3));
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
            // A NaN in V at a token that some row does not see must not reach
            // that row through its weight 0: such a chunk (a block behind the
            // sequence's end may hold anything) multiplies with the NaNs taken
            // out and adds them back for the rows that see them.
            bool fix = false;
            if (masked) {
                uint32_t any = 0u;
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int w = 0; w < DPL / 4; ++w) any |= e4m3_nan_mask(vw[x][w]);
                fix = __any_sync(kFull, any != 0u);
            }
#pragma unroll
            for (int w = 0; w < DPL / 4; ++w) {
                uint32_t nan[4] = {0u, 0u, 0u, 0u};
                if (fix) {
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        nan[x] = e4m3_nan_mask(vw[x][w]) >> 7;  // 1 in each NaN's byte
                        vw[x][w] &= ~(nan[x] * 0xffu);
                        nan[x] *= 0x38u;  // 1.0
                    }
                }
#pragma unroll
                for (int hf = 0; hf < 2; ++hf) {
                    const uint32_t sel = hf == 0 ? 0x5140u : 0x7362u;
                    uint32_t a0, a1, a2, a3;
                    e4m3x4_to_h2(__byte_perm(vw[0][w], vw[1][w], sel), a0, a1);
                    e4m3x4_to_h2(__byte_perm(vw[2][w], vw[3][w], sel), a2, a3);
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_f16(o[n][2 * w + hf], a0, a1, a2, a3, pb[n][0], pb[n][1]);
                    if (fix) {
                        e4m3x4_to_h2(__byte_perm(nan[0], nan[1], sel), a0, a1);
                        e4m3x4_to_h2(__byte_perm(nan[2], nan[3], sel), a2, a3);
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            // which of this lane's four tokens row 8n + j sees
                            const int lj = __shfl_sync(kFull, lim[n][0], j >> 1);
                            const int lk = __shfl_sync(kFull, lim[n][1], j >> 1);
                            const int lr = min((j & 1) ? lk : lj, d.len - 1) - tok0;
                            const uint32_t v0 = (2 * t <= lr ? 0x3c00u : 0u) |
                                                (2 * t + 1 <= lr ? 0x3c000000u : 0u);
                            const uint32_t v1 = (2 * t + 8 <= lr ? 0x3c00u : 0u) |
                                                (2 * t + 9 <= lr ? 0x3c000000u : 0u);
                            float c4[4] = {0.f, 0.f, 0.f, 0.f};
                            mma_f16(c4, a0, a1, a2, a3, v0, v1);
#pragma unroll
                            for (int c = 0; c < 4; ++c)
                                if (c4[c] > 0.f) o[n][2 * w + hf][c] = __uint_as_float(0x7fc00000u);
                        }
                    }
                }
            }
        }

        if (ws.seg_end(i, d)) {
            const bool whole = seg_whole_start && (d.k == d.nch - 1);
            const int b = d.u / units_per_b;
            const int uidx = d.u - b * units_per_b;
            const int h = uidx / p.sub_groups;
            const int sg = uidx - h * p.sub_groups;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float lr = l[n][c];
                    lr += __shfl_xor_sync(kFull, lr, 4);
                    lr += __shfl_xor_sync(kFull, lr, 8);
                    lr += __shfl_xor_sync(kFull, lr, 16);
                    const int r = 8 * n + 2 * t + c;
                    if (r >= seg_rows) continue;
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
                        float* slot = p.partials +
                                      (long long)seg_slot * partial_slot_floats(kp.gs, D);
                        float4* dst = reinterpret_cast<float4*>(slot + r * D + DPL * j);
#pragma unroll
                        for (int x = 0; x < MT / 2; ++x)
                            dst[x] = make_float4(o[n][2 * x][c], o[n][2 * x][c + 2],
                                                 o[n][2 * x + 1][c], o[n][2 * x + 1][c + 2]);
                        if (j == 0) {
                            slot[kp.gs * D + r] = m[n][c];
                            slot[kp.gs * D + kp.gs + r] = lr;
                        }
                    }
                }
        }
        __syncwarp();
        // refill: positions up to i + STAGES (stage i % STAGES is free again)
        while (issued <= i + STAGES && issue(issued)) ++issued;
    }
    pdl_trigger();
}

template <typename T, int D, int NT>
Kv8DecodeInfo make_kv8_decode_info() {
    constexpr int W = 4, S = 4;
    Kv8DecodeInfo info;
    info.fn = kv8_decode_kernel<T, D, NT, W, S>;
    info.warps = W;
    info.stages = S;
    info.smem_bytes = Kv8Layout<D, NT, S, W>::kBytes;
    return info;
}

template <typename T>
Kv8DecodeInfo pick_kv8_decode_info(int head_dim, int rows) {
    if (head_dim == 128)
        return rows <= 8    ? make_kv8_decode_info<T, 128, 1>()
               : rows <= 16 ? make_kv8_decode_info<T, 128, 2>()
                            : make_kv8_decode_info<T, 128, 4>();
    return rows <= 8    ? make_kv8_decode_info<T, 64, 1>()
           : rows <= 16 ? make_kv8_decode_info<T, 64, 2>()
                        : make_kv8_decode_info<T, 64, 4>();
}

}  // namespace pkv
