// page_bounds.cu -- the smallest and the largest key of a page, element by element.
//
// A page is worked out anew from its rows 0 .. x % P, x the last slot written to it, not
// updated from its old bounds: the rows of drafts that were taken back and written again
// leave nothing behind, and a call may be repeated.  Minimum and maximum of 16-bit values
// are exact in 16 bits, so two packed instructions take two elements.
//
// A warp takes a (page, KV head): D / 8 lanes a row, 256 / D rows a load.  What bounds it:
// memory for prompts (the rows are read once: 88,000 tokens of 8 heads of 128, 36.4 us,
// 5.7 TB/s with the grid's start and end), latency for the single pages of a step (2.2 us).
#include "selected.cuh"

namespace pkv {
namespace {

constexpr int kWarps = 4;
constexpr int kMaxTile = 64;  // tokens of a CTA

template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
    using V = __nv_bfloat162;
    static __device__ __forceinline__ V pos_inf() { return __float2bfloat162_rn(INFINITY); }
};
template <>
struct Pair<__half> {
    using V = __half2;
    static __device__ __forceinline__ V pos_inf() { return __float2half2_rn(INFINITY); }
};

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) page_bounds_kernel(const BoundsArgs a, int tile) {
    using V = typename Pair<T>::V;
    constexpr int kRowLanes = D / 8;
    constexpr int kRows = 32 / kRowLanes;  // rows a load of the warp covers
    constexpr int kAhead = 8;              // loads in flight
    __shared__ long long s_last[kMaxTile];
    __shared__ int s_n;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.y, P = a.page_size;
    const int first = blockIdx.x * tile;
    if (threadIdx.x == 0) s_n = 0;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    // (counted from the tile's start: a token's number may be up to 2^31 - 2)
    for (int x = threadIdx.x; x < min(tile, a.n_tokens - first); x += kWarps * 32) {
        const int i = first + x;
        const long long s = a.slots[i];
        if (s < 0) continue;
        if (s >= a.n_slots) {
            set_status(a.status, PKV_DEV_BAD_PAGE);
            continue;
        }
        const bool goes_on = i + 1 < a.n_tokens && (s + 1) % P != 0 && a.slots[i + 1] == s + 1;
        if (!goes_on) s_last[atomicAdd(&s_n, 1)] = s;
    }
    __syncthreads();
    const int n = s_n;
    const int sub = lane / kRowLanes, col = lane % kRowLanes;
    for (int it = warp; it < n; it += kWarps) {
        const long long s = s_last[it], page = s / P;
        const int rows = (int)(s - page * P) + 1;
        const T* base = static_cast<const T*>(a.k_pool) + (page * a.n_kv_heads + h) * P * D;
        V lo[4], hi[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            lo[e] = Pair<T>::pos_inf();
            hi[e] = __hneg2(Pair<T>::pos_inf());
        }
        for (int r0 = 0; r0 < rows; r0 += kAhead * kRows) {
            uint4 x[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                // a row behind the last repeats it
                const int r = min(r0 + u * kRows + sub, rows - 1);
                x[u] = *reinterpret_cast<const uint4*>(base + r * D + col * 8);
            }
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const V* v = reinterpret_cast<const V*>(&x[u]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    lo[e] = __hmin2_nan(lo[e], v[e]);
                    hi[e] = __hmax2_nan(hi[e], v[e]);
                }
            }
        }
#pragma unroll
        for (int o = kRowLanes; o < 32; o <<= 1) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                lo[e] = __hmin2_nan(lo[e], __shfl_xor_sync(kFull, lo[e], o));
                hi[e] = __hmax2_nan(hi[e], __shfl_xor_sync(kFull, hi[e], o));
            }
        }
        if (sub < 2) {
            uint4 y;
            V* v = reinterpret_cast<V*>(&y);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = sub == 0 ? lo[e] : hi[e];
            T* out = static_cast<T*>(a.bounds) + ((page * a.n_kv_heads + h) * 2 + sub) * D;
            *reinterpret_cast<uint4*>(out + col * 8) = y;
        }
    }
}

template <typename T>
cudaError_t launch(const BoundsArgs& a, int head_dim, cudaStream_t stream) {
    // a page a warp while tokens are few (each may be a page of its own), more of them
    // a CTA where a page's tokens stand together
    int tile = kWarps;
    while (tile < kMaxTile && (long long)(a.n_tokens / tile) * a.n_kv_heads > 4096) tile *= 2;
    const dim3 grid(1 + (a.n_tokens - 1) / tile, a.n_kv_heads);
    return launch_pdl(head_dim == 128 ? page_bounds_kernel<T, 128> : page_bounds_kernel<T, 64>,
                      grid, dim3(kWarps * 32), 0, stream, a, tile);
}

}  // namespace

cudaError_t launch_page_bounds(const BoundsArgs& a, bool bf16, int head_dim,
                               cudaStream_t stream) {
    return bf16 ? launch<__nv_bfloat16>(a, head_dim, stream) : launch<__half>(a, head_dim, stream);
}

}  // namespace pkv
