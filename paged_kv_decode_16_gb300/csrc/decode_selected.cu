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
// What bounds it: memory, 4 D bytes a token and KV head; a small batch, the latency of
// list -> table -> rows -> merge.
#include <type_traits>

#include "decode_mma.cuh"
#include "selected.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;
constexpr int kStages = 3;

template <int D, bool TWO>
struct SelLayout {
    static constexpr int kRows = TWO ? 16 : 8;                  // query rows kept of a tile
    static constexpr int kBoxes = D / 64;
    static constexpr int kBoxBytes = kChunk * 128;
    static constexpr int kStageBytes = 2 * kBoxes * kBoxBytes;  // K boxes, then V boxes
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    // behind the chunks the ring's memory holds the states: o [rows][D] of each warp and of
    // the CTA, then m and l of each
    static constexpr int kStateFloats = kRows * D;
    static constexpr int kOffBar = kRing;
    static constexpr int kOffML = kOffBar + kWarps * kStages * 8;
    static constexpr int kBytes = kOffML + (kWarps + 1) * 2 * 16 * 4 + 1024;  // + alignment
    static_assert((kWarps + 1) * kStateFloats * 4 <= kRing, "the states fit the ring");
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                     : "memory");
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

template <typename T, int D, bool TWO>
__global__ void __launch_bounds__(kWarps * 32)
selected_kernel(const SelectedParams p, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap) {
    using Lay = SelLayout<D, TWO>;
    constexpr int KSTEPS = D / 16;
    constexpr int NT = D / 8;
    constexpr bool kSplitP = std::is_same<T, __nv_bfloat16>::value;

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
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
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
    int row_a, used_a, row_b, used_b;  // chunks base .. base + 31 and the 32 behind them
    describe(lane, &row_a, &used_a);
    describe(32 + lane, &row_b, &used_b);

    uint32_t qa[KSTEPS][4];  // A fragments of Q (rows g_lo, g_lo + 8)
    {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const T*>(p.q) + q_row * D);
#pragma unroll
        for (int kk = 0; kk < KSTEPS; ++kk) {
            const int c0 = (kk * 16 + tq) / 2, c1 = c0 + 4;
            qa[kk][0] = g_lo < rows ? q[g_lo * (D / 2) + c0] : 0u;
            qa[kk][2] = g_lo < rows ? q[g_lo * (D / 2) + c1] : 0u;
            qa[kk][1] = TWO && g_lo + 8 < rows ? q[(g_lo + 8) * (D / 2) + c0] : 0u;
            qa[kk][3] = TWO && g_lo + 8 < rows ? q[(g_lo + 8) * (D / 2) + c1] : 0u;
        }
    }

    const uint64_t policy = l2_evict_first_policy();
    int base_i = 0;  // row_a is of chunks base_i .. base_i + 31
    auto issue = [&](int i) {
        const int at = i - base_i;  // < 64
        const int ra = __shfl_sync(kFull, row_a, at & 31), rb = __shfl_sync(kFull, row_b, at & 31);
        const int y = at < 32 ? ra : rb;
        if (lane == 0 && y >= 0) {
            const int st = i % kStages;
            uint8_t* stage = ring + st * Lay::kStageBytes;
            fence_proxy_async_smem();
            mbar_arrive_expect_tx(&bar[st], Lay::kStageBytes);
#pragma unroll
            for (int bx = 0; bx < Lay::kBoxes; ++bx) {
                tma_load_2d_hint(stage + bx * Lay::kBoxBytes, &kmap, bx * 64, y, &bar[st], policy);
                tma_load_2d_hint(stage + (Lay::kBoxes + bx) * Lay::kBoxBytes, &vmap, bx * 64, y,
                                 &bar[st], policy);
            }
        } else if (lane == 0) {
            mbar_arrive(&bar[i % kStages]);
        }
    };
    int issued = 0;
    while (issued < kStages && issued < mine) issue(issued++);

    float o[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) o[nt][0] = o[nt][1] = o[nt][2] = o[nt][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    const int mi = lane >> 3, rr = lane & 7;

    for (int i = 0; i < mine; ++i) {
        const int st = i % kStages;
        const int used = __shfl_sync(kFull, used_a, i - base_i);
        if (!mbar_wait_bounded(&bar[st], (uint32_t)((i / kStages) & 1))) {
            // a copy never landed: report it, wait (bounded) for those in flight
            if (lane == 0) set_status(p.status, PKV_DEV_TIMEOUT);
            for (int j = i + 1; j < issued; ++j)
                mbar_wait_bounded(&bar[j % kStages], (uint32_t)((j / kStages) & 1));
            break;
        }
        if (used > 0) {
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
            // S = Q K^T: tokens 0 - 7 and 8 - 15, even and odd k-steps in chains of their own
            float s[2][2][4] = {};
            const int k_tok = (mi >> 1) * 8 + rr;
#pragma unroll
            for (int kk = 0; kk < KSTEPS; ++kk) {
                const int d = kk * 16 + (mi & 1) * 8;
                uint32_t kb[4];
                ldsm_x4(kst + (d / 64) * Lay::kBoxBytes + swz128(k_tok, (d % 64) / 8), kb);
                Mma<T>::run(s[0][kk & 1], qa[kk], kb[0], kb[1]);
                Mma<T>::run(s[1][kk & 1], qa[kk], kb[2], kb[3]);
            }
            uint32_t pa[4] = {0u, 0u, 0u, 0u}, pl[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int half = 0; half < (TWO ? 2 : 1); ++half) {
                float sc[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int a = e >> 1, x = 2 * half + (e & 1);
                    const int tok = a * 8 + tq + (e & 1);
                    sc[e] = tok < used ? (s[a][0][x] + s[a][1][x]) * p.scale_log2 : -INFINITY;
                }
                float mx = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
                const float m_new = fmaxf(m[half], mx);
                const float ref = m_new == -INFINITY ? 0.f : m_new;
                const float alpha = fast_exp2(m[half] - ref);
                float e[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) e[x] = fast_exp2(sc[x] - ref);
                float sum = (e[0] + e[1]) + (e[2] + e[3]);
                sum += __shfl_xor_sync(kFull, sum, 1);
                sum += __shfl_xor_sync(kFull, sum, 2);
                l[half] = l[half] * alpha + sum;
                m[half] = m_new;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    o[nt][2 * half] *= alpha;
                    o[nt][2 * half + 1] *= alpha;
                }
                if constexpr (kSplitP) {
                    split_bf16x2(e[0], e[1], pa[half], pl[half]);
                    split_bf16x2(e[2], e[3], pa[2 + half], pl[2 + half]);
                } else {
                    pa[half] = Cvt<T>::pack2(e[0], e[1]);
                    pa[2 + half] = Cvt<T>::pack2(e[2], e[3]);
                }
            }
            // O += P V; P in bf16 as a high part and the rest, two products
            const int v_tok = (mi & 1) * 8 + rr;
#pragma unroll
            for (int np = 0; np < NT / 2; ++np) {
                const int d = np * 16 + (mi >> 1) * 8;
                uint32_t vb[4];
                ldsm_x4_trans(vst + (d / 64) * Lay::kBoxBytes + swz128(v_tok, (d % 64) / 8), vb);
                Mma<T>::run(o[2 * np], pa, vb[0], vb[1]);
                Mma<T>::run(o[2 * np + 1], pa, vb[2], vb[3]);
                if constexpr (kSplitP) {
                    Mma<T>::run(o[2 * np], pl, vb[0], vb[1]);
                    Mma<T>::run(o[2 * np + 1], pl, vb[2], vb[3]);
                }
            }
        }
        __syncwarp();
        if (issued < mine) issue(issued++);
        if (i + 1 - base_i == 32) {
            base_i += 32;
            row_a = row_b;
            used_a = used_b;
            describe(base_i + 32 + lane, &row_b, &used_b);
        }
    }
    if (bits) set_status(p.status, bits);

    // ---- the warps' states, in the ring's memory (every copy has been waited for) ----
    __syncthreads();
#pragma unroll
    for (int half = 0; half < (TWO ? 2 : 1); ++half) {
        const int g = g_lo + half * 8;
        float* dst = s_o + warp * Lay::kStateFloats + g * D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            *reinterpret_cast<float2*>(dst + nt * 8 + tq) =
                make_float2(o[nt][2 * half], o[nt][2 * half + 1]);
        if ((lane & 3) == 0) {
            s_m[warp * 32 + g] = m[half];
            s_m[warp * 32 + 16 + g] = l[half];
        }
    }
    __syncthreads();
    T* out = static_cast<T*>(p.out) + q_row * D;
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
            const float4 x =
                *reinterpret_cast<const float4*>(s_o + w * Lay::kStateFloats + g * D + c);
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
            *reinterpret_cast<float4*>(s_o + kWarps * Lay::kStateFloats + g * D + c) = acc;
            if (c == 0) {
                s_m[kWarps * 32 + g] = top;
                s_m[kWarps * 32 + 16 + g] = sum;
            }
        }
    }
    if (ranks == 1) return;
    // ---- the CTAs' states: each CTA writes its share of the outputs ----
    cluster_sync();
    const uint32_t my_o = smem_u32(s_o + kWarps * Lay::kStateFloats);
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
            const float4 x = peer_load4(peer_addr(my_o + (g * D + c) * 4, r));
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
    cluster_sync();  // no CTA leaves while another one reads its memory
}

template <typename T, int D, bool TWO>
cudaError_t launch(const SelectedParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                   cudaStream_t stream) {
    constexpr int kBytes = SelLayout<D, TWO>::kBytes;
    auto kernel = selected_kernel<T, D, TWO>;
    cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
        return e;
    // CTAs of a unit: a wave of two CTAs an SM, while a warp keeps two chunks
    const long long units = (long long)p.batch * p.n_kv_heads * p.head_blocks;
    const long long pages = p.max_pages < p.table_stride ? p.max_pages : p.table_stride;
    const long long chunks = pages * (p.page_size / kChunk);
    int ranks = 1;
    while (ranks < 8 && units * ranks < 2 * sms && chunks >= 2LL * kWarps * 2 * ranks) ranks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(units * ranks));
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

template <typename T>
cudaError_t pick(const SelectedParams& p, int head_dim, const CUtensorMap& kmap,
                 const CUtensorMap& vmap, cudaStream_t stream) {
    const bool two = p.group > 8;
    if (head_dim == 128)
        return two ? launch<T, 128, true>(p, kmap, vmap, stream)
                   : launch<T, 128, false>(p, kmap, vmap, stream);
    return two ? launch<T, 64, true>(p, kmap, vmap, stream)
               : launch<T, 64, false>(p, kmap, vmap, stream);
}

}  // namespace

cudaError_t launch_selected(const SelectedParams& p, bool bf16, int head_dim,
                            const CUtensorMap& kmap, const CUtensorMap& vmap,
                            cudaStream_t stream) {
    return bf16 ? pick<__nv_bfloat16>(p, head_dim, kmap, vmap, stream)
                : pick<__half>(p, head_dim, kmap, vmap, stream);
}

}  // namespace pkv
