// decode_selected.cu -- decode attention over the selected pages of each (request, KV head).
//
// out = sum_t softmax(scale q . k_t) v_t over the tokens t of the listed pages, by the
// running maximum and sum of a softmax, one pass over the data.  The chunk of 16 tokens,
// its two products on the tensor cores (mma.sync: a group's queries are the rows) and its
// tensor copies are those of the plain decode (decode_mma.cuh).  What differs is the work
// split: a list has at most max_pages pages whatever the context, and every request and
// head has the same bound, so there is nothing to plan.  A cluster of CTAs takes one
// (request, KV head, block of 16 query heads); its warps take the list's chunks in turn,
// and the warps' states are merged in shared memory, first within a CTA, then over the
// cluster through distributed shared memory: no workspace, no second launch.
//
// The products are transposed, S^T = K Q^T and O^T = V^T P^T, so that 16 tokens (16 elements
// of the head) fill the 16 rows of an instruction and 8 query heads its 8 columns: half the
// instructions of the form with the heads as rows, of which a group of 8 or less leaves
// half empty.  P^T comes from S^T's accumulators by an 8 x 8 transpose (movmatrix).  P enters
// in two 16-bit pieces, so that it keeps 16 (bf16) or 22 (fp16) significant bits.  fp16's
// range ends at steps of 2^-24, so its weights are taken 2^15 times: the largest, 1, still fits,
// and any is off by 2^-39 of the largest at most.  The first piece is cut, not rounded,
// and the second never 0 beside one that is not: a product with an infinity is then that
// infinity in both, where a rest below 0, or of 0, would make NaN of their sum.
//
// What bounds it: memory, 4 D bytes a token and KV head (256 units of 512 tokens, 134 MB:
// 24 us, 5.6 TB/s, of which 4 are the chain below; 1024 units, 455 MB: 70 us, 6.5 TB/s); a
// small batch, the latency of list -> table -> rows -> merge (3.4 us) and a warp's chunks one
// after another (0.6 to 0.7 us each).
#include <type_traits>

#include "decode_mma.cuh"
#include "selected.cuh"

namespace pkv {
namespace {


template <int D, int HT, int kWarps, int kStages>
struct SelLayout {
    static constexpr int kRows = 8 * HT;                        // query heads of a unit
    static constexpr int kBoxes = D / 64;
    static constexpr int kBoxBytes = kChunk * 128;
    static constexpr int kStageBytes = 2 * kBoxes * kBoxBytes;  // K boxes, then V boxes
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    // behind the chunks the ring's memory holds the states: o [rows][D] of each warp and of
    // the CTA (rows 16 bytes apart: a warp's stores then meet no bank twice), then m and l
    static constexpr int kRowFloats = D + 4;
    static constexpr int kStateFloats = kRows * kRowFloats;
    static constexpr int kOffBar = kRing > (kWarps + 1) * kStateFloats * 4
                                       ? kRing : ((kWarps + 1) * kStateFloats * 4 + 15) / 16 * 16;
    static constexpr int kOffML = kOffBar + kWarps * kStages * 8;
    static constexpr int kBytes = kOffML + (kWarps + 1) * 2 * 16 * 4 + 1024;  // + alignment
};

// The 8 x 8 matrix of 16-bit values that a warp holds (lane l: row l / 4, columns 2 (l % 4)
// and the next), transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// The shared-memory address `addr` of this CTA in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float peer_load(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 peer_load4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// P (>= 0) in two fp16 pieces, kHalfScale times P: cut at 11 bits, and 11 bits of the rest, at
// least fp16's smallest step (2^-24) where the first piece is that much.
constexpr float kHalfScale = 32768.f;
__device__ __forceinline__ void split_cut(__half, float a, float b, uint32_t& hi, uint32_t& lo) {
    a *= kHalfScale;
    b *= kHalfScale;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
    const __half2 h = *reinterpret_cast<const __half2*>(&hi);
    const float2 f = __half22float2(h);
    const __half2 rest = __floats2half2_rn(a - f.x, b - f.y);
    const __half2_raw step = {1, 1};
    const __half2 l = __hmax2(rest, __hmin2(h, __half2(step)));
    lo = *reinterpret_cast<const uint32_t*>(&l);
}
// In two bf16 pieces: cut at 8 bits (the upper half of its bits), and 8 bits of the rest, which
// 2^-23 of P keep above 0.
__device__ __forceinline__ void split_cut(__nv_bfloat16, float a, float b, uint32_t& hi,
                                          uint32_t& lo) {
    hi = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
    const float ha = __uint_as_float(hi << 16), hb = __uint_as_float(hi & 0xffff0000u);
    constexpr float kMore = 1.00000011920928955f;  // 1 + 2^-23
    lo = Cvt<__nv_bfloat16>::pack2(fmaf(a, kMore, -ha), fmaf(b, kMore, -hb));
}

template <typename T, int D, int HT, int kWarps, int kStages>
__global__ void __launch_bounds__(kWarps * 32, kWarps == 8 ? 1 : 2)
selected_kernel(const SelectedParams p, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
    using Lay = SelLayout<D, HT, kWarps, kStages>;
    constexpr int KSTEPS = D / 16;
    constexpr int DT = D / 16;  // tiles of the output
    // o holds fp16's P scaled
    constexpr float kOnce = std::is_same<T, __half>::value ? 1.f / kHalfScale : 1.f;

    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t pad = ((raw + 1023u) & ~1023u) - raw;
    uint8_t* base = smem_raw + pad;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* ring = base + warp * kStages * Lay::kStageBytes;
    const uint32_t ring_u32 = smem_u32(ring);
    uint64_t* bar = reinterpret_cast<uint64_t*>(base + Lay::kOffBar) + warp * kStages;
    float* s_o = reinterpret_cast<float*>(base);               // [warps + 1][rows][D]
    float* s_m = reinterpret_cast<float*>(base + Lay::kOffML);  // [warps + 1][2][16]

    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < kStages; ++s) mbar_init(&bar[s], 1);
        fence_barrier_init();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap))
                     : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap))
                     : "memory");
    }
    __syncwarp();
    const int rank = (int)cluster_rank(), ranks = (int)cluster_size();
    const int unit = blockIdx.x / ranks;
    const int hb = unit % p.head_blocks;
    const int h = unit / p.head_blocks % p.n_kv_heads;
    const int b = unit / p.head_blocks / p.n_kv_heads;
    const int rows = min(p.group - hb * 16, 16);  // query heads of this block
    const long long q_row = (long long)b * p.n_q_heads + h * p.group + hb * 16;
    const int P = p.page_size, per_page = P / kChunk;
    const int g_lo = lane >> 2, tq = (lane & 3) * 2;
    pdl_wait();
    pdl_trigger();

    int len = p.lens[b];
    const long long cap = (long long)p.table_stride * P;
    uint32_t bits = 0;
    if (len < 0 || len > cap) {
        bits = PKV_DEV_BAD_LEN;
        len = len < 0 ? 0 : (int)cap;
    }
    const int n_pages = (int)(((long long)len + P - 1) / P);
    const int32_t* list = p.selected + ((long long)b * p.n_kv_heads + h) * p.max_pages;
    const int32_t* table = p.table + (long long)b * p.table_stride;

    // This warp's chunks: worker, worker + workers, ... of the list's.  A lane works out
    // one of the next 32: its first pool row (-1: nothing there) and tokens in use.
    const int workers = ranks * kWarps, worker = rank * kWarps + warp;
    const long long chunks = (long long)p.max_pages * per_page;
    const int mine = chunks > worker ? (int)((chunks - worker + workers - 1) / workers) : 0;
    auto describe = [&](int i, int* row, int* used) {
        *row = -1;
        *used = 0;
        if (i >= mine) return;
        const long long c = (long long)i * workers + worker;
        const int e = (int)(c / per_page), part = (int)(c - (long long)e * per_page);
        const int s = list[e];
        if (s < 0) return;
        if (s >= n_pages || (e > 0 && s <= list[e - 1])) {
            bits |= PKV_DEV_BAD_LEN;
            return;
        }
        const int page = table[s];
        if (page < 0 || page >= p.num_pages) {
            bits |= PKV_DEV_BAD_PAGE;
            return;
        }
        const long long left = (long long)len - ((long long)s * P + part * kChunk);
        if (left <= 0) return;
        *row = (int)(((long long)page * p.n_kv_heads + h) * P + part * kChunk);
        *used = (int)min(left, (long long)kChunk);
    };
    int row_a, used_a, row_b, used_b;  // the 32 chunks from `at` on and the 32 behind them
    describe(lane, &row_a, &used_a);
    describe(32 + lane, &row_b, &used_b);

    uint32_t qb[HT][KSTEPS][2];  // B fragments of Q^T: heads as columns
    {
        const uint32_t* q =
            reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.q) + q_row * D);
#pragma unroll
        for (int ht = 0; ht < HT; ++ht)
#pragma unroll
            for (int kk = 0; kk < KSTEPS; ++kk) {
                const int at = (8 * ht + g_lo) * (D / 2) + (kk * 16 + tq) / 2;
                const bool in = 8 * ht + g_lo < rows;
                qb[ht][kk][0] = in ? q[at] : 0u;
                qb[ht][kk][1] = in ? q[at + 4] : 0u;
            }
    }

    const uint64_t policy = l2_evict_first_policy();
    int at = 0, issued = 0;
    uint32_t todo = __ballot_sync(kFull, row_a >= 0);  // chunks of row_a not on their way yet
    uint32_t used_st = 0;                              // tokens in use of each stage, 5 bits each
    // Bring in the next chunk that has tokens; false when there is none.
    auto issue = [&]() {
        while (todo == 0) {
            at += 32;
            if (at >= mine) return false;
            row_a = row_b;
            used_a = used_b;
            todo = __ballot_sync(kFull, row_a >= 0);
            describe(at + 32 + lane, &row_b, &used_b);
        }
        const int from = __ffs(todo) - 1, st = issued % kStages;
        todo &= todo - 1;
        const int y = __shfl_sync(kFull, row_a, from), used = __shfl_sync(kFull, used_a, from);
        used_st = (used_st & ~(31u << 5 * st)) | (uint32_t)used << 5 * st;
        if (lane == 0) {
            uint8_t* stage = ring + st * Lay::kStageBytes;
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(&bar[st], Lay::kStageBytes);
#pragma unroll
            for (int bx = 0; bx < Lay::kBoxes; ++bx) {
                tma_load_2d_hint(stage + bx * Lay::kBoxBytes, &kmap, bx * 64, y, &bar[st], policy);
                tma_load_2d_hint(stage + (Lay::kBoxes + bx) * Lay::kBoxBytes, &vmap, bx * 64, y,
                                 &bar[st], policy);
            }
        }
        ++issued;
        return true;
    };
    while (issued < kStages && issue()) {
    }

    // O^T: rows d = 16 dt + g_lo and + 8, columns heads 8 ht + tq and + 1.  m: the maxima of
    // those two heads, l: this lane's part of their sums.
    float o[HT][DT][4];
    float m[HT][2], l[HT][2];
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
#pragma unroll
        for (int dt = 0; dt < DT; ++dt)
            o[ht][dt][0] = o[ht][dt][1] = o[ht][dt][2] = o[ht][dt][3] = 0.f;
        m[ht][0] = m[ht][1] = -INFINITY;
        l[ht][0] = l[ht][1] = 0.f;
    }
    const int mi = lane >> 3, rr = lane & 7;

    for (int i = 0; i < issued; ++i) {
        const int st = i % kStages;
        const int used = (int)(used_st >> 5 * st & 31u);
        if (!mbar_wait_bounded(&bar[st], (uint32_t)((i / kStages) & 1))) {
            // a copy never landed: report it, wait (bounded) for those in flight
            if (lane == 0) set_status(p.status, PKV_DEV_TIMEOUT);
            for (int j = i + 1; j < issued; ++j)
                mbar_wait_bounded(&bar[j % kStages], (uint32_t)((j / kStages) & 1));
            break;
        }
        const uint32_t kst = ring_u32 + st * Lay::kStageBytes;
        const uint32_t vst = kst + Lay::kBoxes * Lay::kBoxBytes;
        if (used < kChunk) {
            // V rows behind the sequence's end may hold anything
            uint4* v = reinterpret_cast<uint4*>(ring + st * Lay::kStageBytes +
                                                Lay::kBoxes * Lay::kBoxBytes);
            for (int z = lane; z < (kChunk - used) * 8 * Lay::kBoxes; z += 32) {
                const int bx = z / ((kChunk - used) * 8), rem = z - bx * (kChunk - used) * 8;
                v[(bx * Lay::kBoxBytes + (used + rem / 8) * 128) / 16 + (rem & 7)] =
                    make_uint4(0u, 0u, 0u, 0u);
            }
            __syncwarp();
        }
        // S^T = K Q^T: tokens are the rows, even and odd k-steps in chains of their own
        float s[HT][2][4] = {};
#pragma unroll
        for (int kk = 0; kk < KSTEPS; ++kk) {
            const int d = kk * 16 + (mi >> 1) * 8;
            uint32_t ka[4];
            ldsm_x4(kst + (d / 64) * Lay::kBoxBytes + swz128((mi & 1) * 8 + rr, (d % 64) / 8), ka);
#pragma unroll
            for (int ht = 0; ht < HT; ++ht)
                Mma<T>::run(s[ht][kk & 1], ka, qb[ht][kk][0], qb[ht][kk][1]);
        }
        uint32_t pb[HT][2], pl[HT][2];  // B fragments of P^T's two pieces
#pragma unroll
        for (int ht = 0; ht < HT; ++ht) {
            float e[4], alpha[2];  // e: (token g_lo, heads tq, tq + 1), (token g_lo + 8, ..)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float v = (s[ht][0][x] + s[ht][1][x]) * p.scale_log2;
                e[x] = g_lo + (x & 2) * 4 < used ? v : -INFINITY;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float mx = fmaxf(e[c], e[2 + c]);
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
                const float m_new = fmaxf(m[ht][c], mx);
                const float ref = m_new == -INFINITY ? 0.f : m_new;
                alpha[c] = fast_exp2(m[ht][c] - ref);
                e[c] = fast_exp2(e[c] - ref);
                e[2 + c] = fast_exp2(e[2 + c] - ref);
                l[ht][c] = fmaf(l[ht][c], alpha[c], e[c] + e[2 + c]);
                m[ht][c] = m_new;
            }
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                o[ht][dt][0] *= alpha[0];
                o[ht][dt][1] *= alpha[1];
                o[ht][dt][2] *= alpha[0];
                o[ht][dt][3] *= alpha[1];
            }
            split_cut(T(), e[0], e[1], pb[ht][0], pl[ht][0]);
            split_cut(T(), e[2], e[3], pb[ht][1], pl[ht][1]);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                pb[ht][x] = transpose8(pb[ht][x]);
                pl[ht][x] = transpose8(pl[ht][x]);
            }
        }
        // O^T += V^T P^T, P as a high part and the rest: two products
#pragma unroll
        for (int dt = 0; dt < DT; ++dt) {
            const int d = dt * 16 + (mi & 1) * 8;
            uint32_t va[4];
            const int tok = (mi >> 1) * 8 + rr;
            ldsm_x4_trans(vst + (d / 64) * Lay::kBoxBytes + swz128(tok, (d % 64) / 8), va);
#pragma unroll
            for (int ht = 0; ht < HT; ++ht) {
                Mma<T>::run(o[ht][dt], va, pb[ht][0], pb[ht][1]);
                Mma<T>::run(o[ht][dt], va, pl[ht][0], pl[ht][1]);
            }
        }
        __syncwarp();
        issue();
    }
    if (bits) set_status(p.status, bits);

    // ---- the warps' states, in the ring's memory (every copy has been waited for) ----
    __syncthreads();
#pragma unroll
    for (int ht = 0; ht < HT; ++ht) {
        const int g = 8 * ht + tq;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float* dst = s_o + warp * Lay::kStateFloats + (g + c) * Lay::kRowFloats + g_lo;
#pragma unroll
            for (int dt = 0; dt < DT; ++dt) {
                dst[dt * 16] = o[ht][dt][c] * kOnce;
                dst[dt * 16 + 8] = o[ht][dt][2 + c] * kOnce;
            }
            float sum = l[ht][c];
            sum += __shfl_xor_sync(kFull, sum, 4);
            sum += __shfl_xor_sync(kFull, sum, 8);
            sum += __shfl_xor_sync(kFull, sum, 16);
            if (g_lo == 0) {
                s_m[warp * 32 + g + c] = m[ht][c];
                s_m[warp * 32 + 16 + g + c] = sum;
            }
        }
    }
    __syncthreads();
    T* out = static_cast<T*>(p.out) + q_row * D;
    float* s_cta = s_o + kWarps * Lay::kStateFloats;  // the CTA's state
    auto weight = [](float m, float top) {  // of a state with maximum m among maxima up to top
        return m == -INFINITY ? 0.f : fast_exp2(m - top);
    };
    for (int z = threadIdx.x; z < rows * (D / 4); z += kWarps * 32) {
        const int g = z / (D / 4), c = z % (D / 4) * 4;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w * 32 + g]);
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = weight(s_m[w * 32 + g], top);
            const float4 x = *reinterpret_cast<const float4*>(s_o + w * Lay::kStateFloats +
                                                              g * Lay::kRowFloats + c);
            sum = fmaf(f, s_m[w * 32 + 16 + g], sum);
            acc.x = fmaf(f, x.x, acc.x);
            acc.y = fmaf(f, x.y, acc.y);
            acc.z = fmaf(f, x.z, acc.z);
            acc.w = fmaf(f, x.w, acc.w);
        }
        if (ranks == 1) {
            const float inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
            *reinterpret_cast<uint2*>(out + g * D + c) = make_uint2(
                Cvt<T>::pack2(acc.x * inv, acc.y * inv), Cvt<T>::pack2(acc.z * inv, acc.w * inv));
        } else {
            *reinterpret_cast<float4*>(s_cta + g * Lay::kRowFloats + c) = acc;
            if (c == 0) {
                s_m[kWarps * 32 + g] = top;
                s_m[kWarps * 32 + 16 + g] = sum;
            }
        }
    }
    if (ranks == 1) return;
    // ---- the CTAs' states: each CTA writes its share of the outputs ----
    cluster_arrive();
    cluster_wait();
    const uint32_t my_o = smem_u32(s_cta);
    const uint32_t my_m = smem_u32(s_m + kWarps * 32);
    for (int z = rank * kWarps * 32 + threadIdx.x; z < rows * (D / 4);
         z += ranks * kWarps * 32) {
        const int g = z / (D / 4), c = z % (D / 4) * 4;
        float top = -INFINITY;
        for (int r = 0; r < ranks; ++r) top = fmaxf(top, peer_load(peer_addr(my_m + g * 4, r)));
        float sum = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int r = 0; r < ranks; ++r) {
            const float f = weight(peer_load(peer_addr(my_m + g * 4, r)), top);
            const float4 x = peer_load4(peer_addr(my_o + (g * Lay::kRowFloats + c) * 4, r));
            sum = fmaf(f, peer_load(peer_addr(my_m + (16 + g) * 4, r)), sum);
            acc.x = fmaf(f, x.x, acc.x);
            acc.y = fmaf(f, x.y, acc.y);
            acc.z = fmaf(f, x.z, acc.z);
            acc.w = fmaf(f, x.w, acc.w);
        }
        const float inv = sum > 0.f || sum != sum ? 1.0f / sum : 0.f;
        *reinterpret_cast<uint2*>(out + g * D + c) = make_uint2(
            Cvt<T>::pack2(acc.x * inv, acc.y * inv), Cvt<T>::pack2(acc.z * inv, acc.w * inv));
    }
    cluster_arrive();
    cluster_wait();  // no CTA leaves while another one reads its memory
}

template <typename T, int D, int HT, int kWarps, int kStages>
cudaError_t launch_clusters(const SelectedParams& p, const CUtensorMap& kmap,
                            const CUtensorMap& vmap, int ranks, cudaStream_t stream) {
    constexpr int kBytes = SelLayout<D, HT, kWarps, kStages>::kBytes;
    auto kernel = selected_kernel<T, D, HT, kWarps, kStages>;
    static SmemLimit limit;
    const cudaError_t e = limit.set(reinterpret_cast<const void*>(kernel), kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.batch * p.n_kv_heads * p.head_blocks * ranks);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p, kmap, vmap);
}

// Up to a CTA an SM, the time is that of a warp's chunks one after another: eight warps a
// CTA with three stages each (all of an SM's shared memory), and as many CTAs a unit as fit.
// Beyond it, bytes in flight count, and a second wave costs: six warps with two stages, two
// CTAs an SM.  us a call, bf16, D 128, group 4, eight warps / six: 192 units of 64 chunks
// 19.5 / 18.0, of 16 chunks 8.5 / 6.1; 256 units of 64 chunks 22.2 / 20.0; and against four
// warps (the cluster size that suits each): 8 units of 256 chunks 7.7 / 9.4, 64 units 20.0 /
// 24.6, 152 units 46.2 / 48.9.
template <typename T, int D, int HT>
cudaError_t launch(const SelectedParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                   cudaStream_t stream) {
    const long long units = (long long)p.batch * p.n_kv_heads * p.head_blocks;
    const int sms = sm_count();
    if (units > sms) return launch_clusters<T, D, HT, 6, 2>(p, kmap, vmap, 1, stream);
    const long long pages = p.max_pages < p.table_stride ? p.max_pages : p.table_stride;
    const long long chunks = pages * (p.page_size / kChunk);
    // steps of a warp, and the cluster's merge, which costs about as much as one
    // (8 units of 64 chunks, clusters of 1 / 2 / 4 / 8: 8.9 / 7.0 / 5.6 / 5.3 us; of 16 chunks
    // 4.4 / 4.8 / 4.9 / 5.2)
    int ranks = 1;
    long long best = (chunks + 7) / 8;
    for (int r = 2; r <= 8 && units * r <= sms; r *= 2) {
        const long long steps = (chunks + 8 * r - 1) / (8 * r) + 1;
        if (steps < best) {
            best = steps;
            ranks = r;
        }
    }
    return launch_clusters<T, D, HT, 8, 3>(p, kmap, vmap, ranks, stream);
}

template <typename T>
cudaError_t pick(const SelectedParams& p, int head_dim, const CUtensorMap& kmap,
                 const CUtensorMap& vmap, cudaStream_t stream) {
    const bool two = p.group > 8;
    if (head_dim == 128)
        return two ? launch<T, 128, 2>(p, kmap, vmap, stream)
                   : launch<T, 128, 1>(p, kmap, vmap, stream);
    return two ? launch<T, 64, 2>(p, kmap, vmap, stream)
               : launch<T, 64, 1>(p, kmap, vmap, stream);
}

}  // namespace

cudaError_t launch_selected(const SelectedParams& p, bool bf16, int head_dim,
                            const CUtensorMap& kmap, const CUtensorMap& vmap,
                            cudaStream_t stream) {
    return bf16 ? pick<__nv_bfloat16>(p, head_dim, kmap, vmap, stream)
                : pick<__half>(p, head_dim, kmap, vmap, stream);
}

}  // namespace pkv
