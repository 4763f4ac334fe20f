// kv8_plan.cuh -- the ranges of the 8-bit cache's attention kernels, worked out by
// every CTA for itself.
#pragma once

#include "kv8.cuh"

namespace pkv {

// The ranges of the whole batch by one CTA: prefix sums into s_prefix, and the
// positions' total.  CTA 0 leaves them in the workspace for the combine kernel.
template <int THREADS>
__device__ __forceinline__ int kv8_self_plan(const Kv8DecodeParams& p, int32_t* s_prefix,
                                             uint32_t* flags) {
    constexpr int PER = (kKv8SelfPlan + THREADS - 1) / THREADS, NWARPS = THREADS / 32;
    __shared__ long long s_tot[NWARPS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int cnt[PER];
    long long sum = 0;
#pragma unroll
    for (int x = 0; x < PER; ++x) {
        const int b = tid * PER + x;
        long long len = b < p.batch ? p.lens[b] : 0;
        if (len < 0 || len > p.cap) {
            if (blockIdx.x == 0) *flags |= PKV_DEV_BAD_LEN;
            len = len < 0 ? 0 : p.cap;
        }
        const int nch = (int)((len + kChunk - 1) / kChunk);
        const long long c = nch ? (long long)(nch + p.unit_cost) * p.units_per_b : 0;
        cnt[x] = (int)c;  // (beyond an int: so is the total, and nothing is done)
        sum += c;
    }
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(kFull, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) s_tot[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NWARPS; ++w) {
        if (w < warp) before += s_tot[w];
        total += s_tot[w];
    }
    if (total > 0x7fffffffLL) {  // beyond the 32-bit positions: refuse the work
        if (blockIdx.x == 0) *flags |= PKV_DEV_BAD_LEN;
        total = 0;
    }
    long long at = before + incl - sum;
#pragma unroll
    for (int x = 0; x < PER; ++x) {
        const int b = tid * PER + x;
        const int v = total ? (int)at : 0;
        if (b <= p.batch) {
            s_prefix[b] = v;
            if (blockIdx.x == 0) p.prefix[b] = v;
        }
        at += cnt[x];
    }
    if (PER * THREADS == kKv8SelfPlan && tid == THREADS - 1 && p.batch == kKv8SelfPlan) {
        s_prefix[kKv8SelfPlan] = (int)total;
        if (blockIdx.x == 0) p.prefix[kKv8SelfPlan] = (int)total;
    }
    __syncthreads();
    return (int)total;
}

}  // namespace pkv
