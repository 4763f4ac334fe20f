// kv8_combine.cu -- merging the partial states of the 8-bit cache's decode.
//
// One CTA per unit, or per (unit, row) when units are few beside the workers
// (their rows have many segments then); units that one worker finished exit at
// once.  The arithmetic is merge.cuh's.  One CTA more than those collects the
// workers' status bits.  What bounds it: two dependent rounds of loads after
// the decode kernel's end; its launch itself overlaps that kernel's tail.
#include "kv8.cuh"
#include "merge.cuh"

namespace pkv {

namespace {

template <typename T, int D>
__global__ void __launch_bounds__(kMergeSlots * 32)
kv8_combine_kernel(const __grid_constant__ Kv8CombineArgs a, int row_split) {
    pdl_wait();  // everything read below, the ranges too, is the decode kernel's
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if ((int)blockIdx.x == a.units * row_split) {
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
    const int u = blockIdx.x / row_split;
    const int part = blockIdx.x - u * row_split;
    const int b = u / a.units_per_b;
    const int uidx = u - b * a.units_per_b;
    const int h = uidx / a.sub_groups;
    const int sg = uidx - h * a.sub_groups;
    const int first = a.prefix[b];
    const int per_unit = (a.prefix[b + 1] - first) / a.units_per_b;
    if (per_unit == 0) return;  // no tokens: the decode kernel wrote zeros
    const UnitSegments segs =
        unit_segments(a.hdr->chunks_per_worker, a.hdr->extra_chunks, u,
                      first + uidx * per_unit + a.unit_cost, per_unit - a.unit_cost);
    const int ns = segs.count();
    if (ns <= 1) return;  // finished in place by its worker
    const int nrows = a.rows.rows(sg);
    if (row_split > 1 && part >= nrows) return;
    const SlotSegs slots{a.partials, segs.base, partial_slot_floats(a.gs, D), a.gs, D};
    T* out = static_cast<T*>(a.out);
    if (row_split > 1) {
        const RowShift<SlotSegs> one{slots, part};
        merge_rows_cta<T, D>(one, ns, 1, warp, lane,
                             [&](int) { return out + a.rows.row(b, h, sg, part) * D; });
    } else {
        merge_rows_cta<T, D>(slots, ns, nrows, warp, lane,
                             [&](int g) { return out + a.rows.row(b, h, sg, g) * D; });
    }
}

}  // namespace

cudaError_t launch_kv8_combine(bool bf16, int head_dim, const Kv8CombineArgs& a, int workers,
                               cudaStream_t stream) {
    const int row_split = (long long)a.units * 32 < workers ? a.gs : 1;
    const dim3 grid((unsigned)((long long)a.units * row_split + 1));
#define PKV_KV8_COMBINE(T, D) \
    return launch_pdl(kv8_combine_kernel<T, D>, grid, dim3(kMergeSlots * 32), 0, stream, a, row_split)
    if (bf16) {
        if (head_dim == 128) PKV_KV8_COMBINE(__nv_bfloat16, 128);
        PKV_KV8_COMBINE(__nv_bfloat16, 64);
    }
    if (head_dim == 128) PKV_KV8_COMBINE(__half, 128);
    PKV_KV8_COMBINE(__half, 64);
#undef PKV_KV8_COMBINE
}

}  // namespace pkv
