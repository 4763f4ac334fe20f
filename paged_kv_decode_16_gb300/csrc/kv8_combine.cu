// kv8_combine.cu -- merging the partial states of the 8-bit cache's decode.
//
// A warp per row of a unit; when units are few beside the workers (their rows
// have many segments then), a CTA per row, whose warps share the segments
// (merge.cuh).  Rows that one worker finished end at once.  A warp's loads --
// every segment's maximum and sum, and the weighted sums of the first eight
// segments -- go out together, before the first of them is used: one round of
// loads behind the one for the ranges is what the kernel takes.  CTA 0 collects
// the workers' status bits.  (A CTA of 8 warps per unit took 5.3 us of a
// decode over 32 sequences of 512 to 4096 tokens and 13 us of one over 256
// uneven ones, whose 1024 CTAs came in three waves.)
#include "kv8.cuh"
#include "merge.cuh"

namespace pkv {

namespace {

constexpr int kBlock = 8;  // segments whose sums are in flight together

// The row's segments by one warp: lane x takes elements 4x .. 4x + 3.
template <typename T, int D>
__device__ __forceinline__ void merge_row_warp(const SlotSegs& sg, int ns, int g, int lane,
                                               T* out) {
    const bool act = lane < D / 4;
    float4 v[kBlock];
#pragma unroll
    for (int x = 0; x < kBlock; ++x)
        if (act && x < ns) v[x] = __ldcg(sg.o4(x, g, lane));
    float M = -INFINITY;
    float m0 = -INFINITY, l0 = 0.f;  // segment `lane`
    if (lane < ns) {
        m0 = __ldcg(sg.m(lane, g));
        l0 = __ldcg(sg.l(lane, g));
    }
    M = m0;
    for (int s = 32 + lane; s < ns; s += 32) M = fmaxf(M, __ldcg(sg.m(s, g)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
    float w = merge_weight(m0, M);
    float den = w * l0;
    for (int s = 32 + lane; s < ns; s += 32)
        den = fmaf(merge_weight(__ldcg(sg.m(s, g)), M), __ldcg(sg.l(s, g)), den);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(kFull, den, o);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int s0 = 0; s0 < ns; s0 += kBlock) {
        if (s0 > 0) {
#pragma unroll
            for (int x = 0; x < kBlock; ++x)
                if (act && s0 + x < ns) v[x] = __ldcg(sg.o4(s0 + x, g, lane));
            // weights of the next 32 segments
            if ((s0 & 31) == 0)
                w = s0 + lane < ns ? merge_weight(__ldcg(sg.m(s0 + lane, g)), M) : 0.f;
        }
#pragma unroll
        for (int x = 0; x < kBlock; ++x) {
            const float ws = __shfl_sync(kFull, w, (s0 + x) & 31);
            if (act && s0 + x < ns) {
                acc.x = fmaf(ws, v[x].x, acc.x);
                acc.y = fmaf(ws, v[x].y, acc.y);
                acc.z = fmaf(ws, v[x].z, acc.z);
                acc.w = fmaf(ws, v[x].w, acc.w);
            }
        }
    }
    if (act) {
        // a sum of 0: no token seen.  (Sums may be as small as 2^-40 and NaN
        // stays NaN, so it is compared with 0.)
        const float inv = den == 0.f ? 0.f : 1.0f / den;
        *reinterpret_cast<uint2*>(out + lane * 4) =
            make_uint2(Cvt<T>::pack2(acc.x * inv, acc.y * inv),
                       Cvt<T>::pack2(acc.z * inv, acc.w * inv));
    }
}

// kRowCta: a CTA per row, else a warp.
template <typename T, int D, bool kRowCta>
__global__ void __launch_bounds__(kMergeSlots * 32)
kv8_combine_kernel(const __grid_constant__ Kv8CombineArgs a) {
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
                                   : ((long long)blockIdx.x - 1) * kMergeSlots + warp;
    const int u = (int)(item / a.gs), g = (int)(item - (long long)u * a.gs);
    if (u >= a.units) return;
    const int b = u / a.units_per_b;
    const int uidx = u - b * a.units_per_b;
    const int h = uidx / a.sub_groups;
    const int sg = uidx - h * a.sub_groups;
    const int first = a.prefix[b], next = a.prefix[b + 1];
    const int sw = a.hdr->chunks_per_worker, r = a.hdr->extra_chunks;
    if (g >= a.rows.rows(sg)) return;
    const int per_unit = (next - first) / a.units_per_b;
    if (per_unit == 0) return;  // no tokens: the decode kernel wrote zeros
    const UnitSegments segs = unit_segments(sw, r, u, first + uidx * per_unit + a.unit_cost,
                                            per_unit - a.unit_cost);
    const int ns = segs.count();
    if (ns <= 1) return;  // finished in place by its worker
    const SlotSegs slots{a.partials, segs.base, partial_slot_floats(a.gs, D), a.gs, D};
    T* out = static_cast<T*>(a.out) + a.rows.row(b, h, sg, g) * D;
    if constexpr (kRowCta) {
        const RowShift<SlotSegs> one{slots, g};
        merge_rows_cta<T, D>(one, ns, 1, warp, lane, [&](int) { return out; });
    } else {
        merge_row_warp<T, D>(slots, ns, g, lane, out);
    }
}

}  // namespace

cudaError_t launch_kv8_combine(bool bf16, int head_dim, const Kv8CombineArgs& a, int workers,
                               cudaStream_t stream) {
    const long long rows = (long long)a.units * a.gs;
    const bool row_cta = (long long)a.units * 32 < workers;
    const long long ctas = 1 + (row_cta ? rows : (rows + kMergeSlots - 1) / kMergeSlots);
    if (ctas > 0x7fffffffLL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)ctas);
#define PKV_KV8_COMBINE(T, D)                                                                  \
    return row_cta ? launch_pdl(kv8_combine_kernel<T, D, true>, grid, dim3(kMergeSlots * 32), 0, \
                                stream, a)                                                      \
                   : launch_pdl(kv8_combine_kernel<T, D, false>, grid, dim3(kMergeSlots * 32),  \
                                0, stream, a)
    if (bf16) {
        if (head_dim == 128) PKV_KV8_COMBINE(__nv_bfloat16, 128);
        PKV_KV8_COMBINE(__nv_bfloat16, 64);
    }
    if (head_dim == 128) PKV_KV8_COMBINE(__half, 128);
    PKV_KV8_COMBINE(__half, 64);
#undef PKV_KV8_COMBINE
}

}  // namespace pkv
