// kv8_combine.cu -- merging the partial states of the 8-bit cache's decode, and the
// plan of batches too large for every CTA to work out its own.
//
// A warp per row of a unit; when units are few beside the decode's CTAs (their
// rows have many segments then), a CTA per row, whose warps take every eighth
// segment each and meet in shared memory.  Rows that the decode kernel finished
// end at once.  A warp's loads -- its segments' maxima and sums, and the weighted
// sums of its first six or eight segments -- go out together, before the first of them
// is used: one round of loads behind the one for the ranges is what the kernel
// takes.  CTA 0 collects the workers' status bits.
//
// Segments of a unit (kv8_decode.cuh): one for each of its workers, in slot
// u + w; where kv8_merge_warps says so, the workers of one CTA whose ranges end within the
// unit, or with it, have merged theirs into one, in the slot of the first.
#include "kv8.cuh"
#include "merge.cuh"

namespace pkv {

namespace {

struct Segs {
    int u, w0;    // unit, its first worker
    int chains;   // merged segments
    int count;    // segments: the chains, and the last worker's own if it has one
    int w_last;
    int per;      // workers merged into one (those of a CTA), 1: none are
    __device__ __forceinline__ long long slot(int s) const {
        return (long long)u + (s == 0         ? w0
                               : s < chains   ? (w0 / per + s) * per
                                              : w_last);
    }
};

// The segments of unit u, whose chunks are positions a .. e.
__device__ __forceinline__ Segs kv8_segments(int sw, int r, int u, int a, int e, int per) {
    Segs s;
    s.u = u;
    s.w0 = worker_of(a, sw, r);
    s.w_last = worker_of(e, sw, r);
    const bool own = s.w_last > s.w0 && e + 1 < range_begin(s.w_last + 1, sw, r);
    const int wt = own ? s.w_last - 1 : s.w_last;
    s.per = per;
    s.chains = wt / per - s.w0 / per + 1;
    s.count = s.chains + (own ? 1 : 0);
    return s;
}

constexpr int kWarps = 8;
// Segments whose sums are in flight together, where a warp takes a row: 6, and 4 CTAs
// an SM (us with 8 and 3 / 6 and 4 / 4 and 5: 32 sequences of 512 to 4096 tokens 26.7 /
// 26.9 / 27.4; with 16 query tokens 86.3 / 85.1 / 84.1; 256 of 16 to 8192 66.3 / 66.0 /
// 65.9; 4 of 1000 to 8192, 64 query tokens 55.2 / 54.3 / 54.2); where a CTA does: 8 (one
// sequence of 32768 22.8, with 6 23.3).
constexpr int kRowBlock = 6, kRowCtasSm = 4, kCtaBlock = 8;

// Segments 0 .. n - 1 of a row by one warp, relative to their own largest
// maximum M: lane x has elements 4x .. 4x + 3 of the weighted sum.  at(s): the
// segment's slot; o, m, l: the row's places in a slot.
template <int D, int kBlock, class At>
__device__ __forceinline__ float4 merge_some(const At& at, int n, int o, int m, int l, int lane,
                                             float& M, float& den) {
    const bool act = lane < D / 4;
    float4 v[kBlock];
#pragma unroll
    for (int x = 0; x < kBlock; ++x)
        if (act && x < n) v[x] = __ldcg(reinterpret_cast<const float4*>(at(x) + o) + lane);
    float m0 = -INFINITY, l0 = 0.f;  // segment `lane`
    if (lane < n) {
        m0 = __ldcg(at(lane) + m);
        l0 = __ldcg(at(lane) + l);
    }
    M = m0;
    for (int x = 32 + lane; x < n; x += 32) M = fmaxf(M, __ldcg(at(x) + m));
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, k));
    float w = merge_weight(m0, M);
    den = w * l0;
    for (int x = 32 + lane; x < n; x += 32)
        den = fmaf(merge_weight(__ldcg(at(x) + m), M), __ldcg(at(x) + l), den);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) den += __shfl_xor_sync(kFull, den, k);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int base = 0; base < n; base += 32) {
        const int stop = min(n, base + 32);
        if (base > 0)  // weights of the next 32
            w = base + lane < n ? merge_weight(__ldcg(at(base + lane) + m), M) : 0.f;
        for (int x0 = base; x0 < stop; x0 += kBlock) {
            if (x0 > 0) {
#pragma unroll
                for (int x = 0; x < kBlock; ++x)
                    if (act && x0 + x < stop)
                        v[x] = __ldcg(reinterpret_cast<const float4*>(at(x0 + x) + o) + lane);
            }
#pragma unroll
            for (int x = 0; x < kBlock; ++x) {
                const float wt = __shfl_sync(kFull, w, (x0 - base + x) & 31);
                if (act && x0 + x < stop) {
                    acc.x = fmaf(wt, v[x].x, acc.x);
                    acc.y = fmaf(wt, v[x].y, acc.y);
                    acc.z = fmaf(wt, v[x].z, acc.z);
                    acc.w = fmaf(wt, v[x].w, acc.w);
                }
            }
        }
    }
    return acc;
}

// A sum of 0: no token seen, zeros.  (Sums may be as small as 2^-40, and NaN
// stays NaN.)
template <typename T>
__device__ __forceinline__ void store_row(const float4& acc, float den, int lane, T* out) {
    const float inv = den == 0.f ? 0.f : 1.0f / den;
    *reinterpret_cast<uint2*>(out + lane * 4) =
        make_uint2(Cvt<T>::pack2(acc.x * inv, acc.y * inv),
                   Cvt<T>::pack2(acc.z * inv, acc.w * inv));
}

// A warp a row, whose slots are next to each other as no workers are merged; the
// same for slots in any order (0.4 to 1.3 us more, 32 sequences of 512 to 4096
// tokens); a CTA a row.
enum Form { kWarpRow, kWarpRowMerged, kCtaRow };

template <typename T, int D, Form kForm>
__global__ void __launch_bounds__(kWarps * 32, kForm == kCtaRow ? 1 : kRowCtasSm)
kv8_combine_kernel(const __grid_constant__ Kv8CombineArgs a) {
    constexpr bool kRowCta = kForm == kCtaRow;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();  // everything read below, the ranges too, is the decode kernel's
    pdl_trigger();
    if (blockIdx.x == 0) {
        __shared__ uint32_t s_bits;
        if (threadIdx.x == 0) s_bits = 0;
        __syncthreads();
        uint32_t bits = 0;
        for (int x = threadIdx.x; x < a.n_flags; x += blockDim.x) bits |= a.flags[x];
        bits = __reduce_or_sync(kFull, bits);
        if (lane == 0 && bits) atomicOr(&s_bits, bits);
        __syncthreads();
        if (threadIdx.x == 0) {
            a.hdr->status = s_bits | (a.self_plan ? 0u : a.hdr->status);
            a.hdr->append_slots = 0;
        }
        return;
    }
    const long long item = kRowCta ? (long long)blockIdx.x - 1
                                   : ((long long)blockIdx.x - 1) * kWarps + warp;
    const int u = (int)(item / a.gs), g = (int)(item - (long long)u * a.gs);
    if (u >= a.units) return;
    const int b = u / a.units_per_b;
    const int uidx = u - b * a.units_per_b;
    const int h = uidx / a.sub_groups;
    const int sg = uidx - h * a.sub_groups;
    const int first = a.prefix[b], next = a.prefix[b + 1];
    const int nw = a.hdr->num_workers, sw = a.hdr->chunks_per_worker, r = a.hdr->extra_chunks;
    if (g >= a.rows.rows(sg)) return;
    const int per_unit = (next - first) / a.units_per_b;
    if (per_unit == 0 || nw <= 0) return;  // no tokens: the decode kernel wrote zeros
    const int at = first + uidx * per_unit;
    const Segs segs = kv8_segments(sw, r, u, at + a.unit_cost, at + per_unit - 1,
                                   kv8_merge_warps(a.units, nw, a.merge));
    if (segs.count <= 1) return;  // finished in the decode kernel
    const int stride = partial_slot_floats(a.gs, D);
    T* out = static_cast<T*>(a.out) + a.rows.row(b, h, sg, g) * D;
    if constexpr (kRowCta) {
        __shared__ float4 s_acc[kWarps][D / 4];
        __shared__ float s_m[kWarps], s_den[kWarps];
        float M, den;
        const int n = segs.count > warp ? (segs.count - warp + kWarps - 1) / kWarps : 0;
        const float4 acc = merge_some<D, kCtaBlock>(
            [&](int s) { return a.partials + segs.slot(warp + s * kWarps) * stride; }, n, g * D,
            a.gs * D + g, a.gs * D + a.gs + g, lane, M, den);
        if (lane < D / 4) s_acc[warp][lane] = acc;
        if (lane == 0) {
            s_m[warp] = M;
            s_den[warp] = den;
        }
        __syncthreads();
        if (warp > 0 || lane >= D / 4) return;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
        float total = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float wt = merge_weight(s_m[w], top);
            const float4 y = s_acc[w][lane];
            total = fmaf(wt, s_den[w], total);
            sum.x = fmaf(wt, y.x, sum.x);
            sum.y = fmaf(wt, y.y, sum.y);
            sum.z = fmaf(wt, y.z, sum.z);
            sum.w = fmaf(wt, y.w, sum.w);
        }
        store_row<T>(sum, total, lane, out);
    } else {
        float M, den;
        const float* slots = a.partials + (segs.u + segs.w0) * (long long)stride;
        const float4 acc = merge_some<D, kRowBlock>(
            [&](int s) {
                return kForm == kWarpRowMerged ? a.partials + segs.slot(s) * stride
                                               : slots + s * stride;
            },
            segs.count, g * D, a.gs * D + g, a.gs * D + a.gs + g, lane, M, den);
        if (lane < D / 4) store_row<T>(acc, den, lane, out);
    }
}

// kv8_plan.cuh's ranges by one CTA, for any batch.
constexpr int kPlanThreads = 1024;

__global__ void __launch_bounds__(kPlanThreads)
kv8_plan_kernel(const __grid_constant__ Kv8DecodeParams p) {
    __shared__ long long s_tot[kPlanThreads / 32];
    __shared__ uint32_t s_bits;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) s_bits = 0;
    pdl_wait();
    long long running = 0;
    uint32_t bits = 0;
    for (int base = 0; base < p.batch; base += kPlanThreads) {
        const int b = base + tid;
        long long len = b < p.batch ? p.lens[b] : 0;
        if (len < 0 || len > p.cap) {
            bits |= PKV_DEV_BAD_LEN;
            len = len < 0 ? 0 : p.cap;
        }
        const long long nch = (len + kChunk - 1) / kChunk;
        const long long c = nch ? (nch + p.unit_cost) * p.units_per_b : 0;
        long long incl = c;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) s_tot[warp] = incl;
        __syncthreads();
        long long before = running;
        for (int w = 0; w < kPlanThreads / 32; ++w) {
            if (w < warp) before += s_tot[w];
            running += s_tot[w];
        }
        if (b < p.batch) p.prefix[b] = (int)(before + incl - c);
        __syncthreads();
    }
    if (running > 0x7fffffffLL) {  // beyond the 32-bit positions: refuse the work
        bits |= PKV_DEV_BAD_LEN;
        running = 0;
    }
    bits = __reduce_or_sync(kFull, bits);
    if (lane == 0 && bits) atomicOr(&s_bits, bits);
    __syncthreads();
    if (tid == 0) {
        int nw, sw, r;
        kv8_ranges((int)running, p.workers_req, p.workers_auto, &nw, &sw, &r);
        p.prefix[p.batch] = (int)running;
        p.hdr->num_workers = nw;
        p.hdr->chunks_per_worker = sw;
        p.hdr->extra_chunks = r;
        p.hdr->status = s_bits;
    }
}

}  // namespace

cudaError_t launch_kv8_plan(const Kv8DecodeParams& p, cudaStream_t stream) {
    return launch_pdl(kv8_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, p);
}

cudaError_t launch_kv8_combine(bool bf16, int head_dim, const Kv8CombineArgs& a, int workers,
                               cudaStream_t stream) {
    const long long rows = (long long)a.units * a.gs;
    // more than about eight segments a unit, if every worker has work (sequences of
    // 4096 tokens, 4 KV heads, group 1: 256 units 48.0 us by warps, 49.6 by CTAs;
    // 128 the same either way)
    const bool row_cta = (long long)a.units * 8 < workers && rows <= kKv8RowCtas;
    const long long ctas = 1 + (row_cta ? rows : (rows + kWarps - 1) / kWarps);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)ctas);
#define PKV_KV8_COMBINE_FORM(T, D, F) \
    return launch_pdl(kv8_combine_kernel<T, D, F>, grid, dim3(kWarps * 32), 0, stream, a)
#define PKV_KV8_COMBINE(T, D)                                      \
    do {                                                           \
        if (row_cta) PKV_KV8_COMBINE_FORM(T, D, kCtaRow);          \
        if (a.merge > 1) PKV_KV8_COMBINE_FORM(T, D, kWarpRowMerged); \
        PKV_KV8_COMBINE_FORM(T, D, kWarpRow);                      \
    } while (0)
    if (bf16) {
        if (head_dim == 128) PKV_KV8_COMBINE(__nv_bfloat16, 128);
        PKV_KV8_COMBINE(__nv_bfloat16, 64);
    }
    if (head_dim == 128) PKV_KV8_COMBINE(__half, 128);
    PKV_KV8_COMBINE(__half, 64);
#undef PKV_KV8_COMBINE
#undef PKV_KV8_COMBINE_FORM
}

}  // namespace pkv
