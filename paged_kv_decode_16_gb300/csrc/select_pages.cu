// select_pages.cu -- the pages that a query attends to: scores, then the choice.
//
// Score of page j for KV head h: max over the head's queries of q+ . hi_j + q- . lo_j, with
// q+ = max(q, 0) and q- = min(q, 0), which is at least q . k for every key of the page.  The
// bounds of a page and head lie as one row [lo | hi] of 2 D elements, so a score is one dot
// product of that row with [q- | q+]: pages are the rows of a matrix product on the
// tensor cores (mma.sync m16n8k16: 16 pages x 8 queries), fed straight from global memory:
// the contraction's order is free, so a lane takes 16 contiguous bytes of a row as its
// fragments of two k-steps.  What bounds it: memory, 4 D bytes a page and head.
//
// The choice is that of exact scores, so that it does not depend on how a product is
// summed.  A product of two 16-bit values is exact in fp32; each of the 2 D / 16 steps adds 16
// of them to the sum, every addend cut at 2^-24 of the largest at worst: 17 addends, 2 D /
// 16 <= 16 steps, so a score is off by at most e = 2^-15 S (S = sum |q_d| max |bound|; the
// count gives 2^-15.9).  The k-th largest score is then off by at most e too: pages more than 2 e above the
// k-th fp32 score are chosen, those more than 2 e below are not, and only the few in
// between are scored again in fp64, where that is not settled by their number.
#include <type_traits>

#include "decode_mma.cuh"
#include "selected.cuh"

namespace pkv {
namespace {

constexpr int kScoreWarps = 4;

__device__ __forceinline__ int pages_of(const SelectArgs& a, int b, uint32_t* bits) {
    int len = a.lens[b];
    const long long cap = (long long)a.table_stride * a.page_size;
    if (len < 0 || len > cap) {
        *bits |= PKV_DEV_BAD_LEN;
        len = len < 0 ? 0 : (int)cap;
    }
    return (int)(((long long)len + a.page_size - 1) / a.page_size);
}

// Largest magnitude of packed 16-bit floats, as bits (NaN above infinity above all).
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t x) {
    return __vmaxu2(m, x & 0x7fff7fffu);
}

template <typename T, int D>
__global__ void __launch_bounds__(kScoreWarps * 32) score_kernel(const SelectArgs a) {
    constexpr int kSegs = 2 * D / 32;           // 64-byte pieces of a row: two k-steps each
    constexpr int kRowBytes = 4 * D + 64;       // a query's [q- | q+], rows 64 bytes apart mod 128
    extern __shared__ __align__(16) uint8_t s_q[];
    __shared__ uint32_t s_max[kScoreWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x, tile = blockIdx.y, b = blockIdx.z;
    const int group = a.n_q_heads / a.n_kv_heads;
    const int rows8 = (group + 7) / 8 * 8;
    pdl_wait();
    pdl_trigger();
    uint32_t bits = 0;
    const int n = pages_of(a, b, &bits);
    const int first = tile * kSelectTile;
    if (bits && h == 0 && tile == 0 && threadIdx.x == 0) set_status(a.status, bits);
    if (n <= a.max_pages || first >= n) return;

    // [q- | q+] of the head's queries; rows behind the group are zeros and not used
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) +
                                                    ((long long)b * a.n_q_heads + h * group) * D);
    for (int i = threadIdx.x; i < rows8 * (D / 8); i += kScoreWarps * 32) {
        const int r = i / (D / 8), c = i % (D / 8);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (r < group) x = q[i];
        uint32_t w[4] = {x.x, x.y, x.z, x.w}, neg[4], pos[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // by the sign bit; a NaN goes to one of the two and makes the score NaN
            const uint32_t sign = (w[e] & 0x80008000u) >> 15;
            const uint32_t mask = sign * 0xffffu;
            neg[e] = w[e] & mask;
            pos[e] = w[e] & ~mask;
        }
        uint8_t* at = s_q + r * kRowBytes + c * 16;
        *reinterpret_cast<uint4*>(at) = make_uint4(neg[0], neg[1], neg[2], neg[3]);
        *reinterpret_cast<uint4*>(at + 2 * D) = make_uint4(pos[0], pos[1], pos[2], pos[3]);
    }
    __syncthreads();

    const int32_t* table = a.table + (long long)b * a.table_stride;
    const T* bounds = static_cast<const T*>(a.bounds);
    const long long unit = (long long)b * a.n_kv_heads + h;
    const int g = lane >> 2, t = lane & 3;
    uint32_t big = 0;
    for (int j0 = first + warp * 16; j0 < min(first + kSelectTile, n); j0 += kScoreWarps * 16) {
        // lanes 0 .. 15 find the pages, every lane then takes rows g and g + 8
        const int j = j0 + (lane & 15);
        int page = j < n ? table[j] : 0;
        bool ok = page >= 0 && page < a.num_pages;
        if (!ok) set_status(a.status, PKV_DEV_BAD_PAGE);
        if (!ok) page = -1;
        const int page0 = __shfl_sync(kFull, page, g), page1 = __shfl_sync(kFull, page, g + 8);
        const bool use0 = j0 + g < n && page0 >= 0, use1 = j0 + g + 8 < n && page1 >= 0;
        uint4 x[kSegs], y[kSegs];
        const uint4* r0 = reinterpret_cast<const uint4*>(
            bounds + ((long long)page0 * a.n_kv_heads + h) * 2 * D);
        const uint4* r1 = reinterpret_cast<const uint4*>(
            bounds + ((long long)page1 * a.n_kv_heads + h) * 2 * D);
#pragma unroll
        for (int s = 0; s < kSegs; ++s) {
            x[s] = use0 ? r0[s * 4 + t] : make_uint4(0, 0, 0, 0);
            y[s] = use1 ? r1[s * 4 + t] : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int s = 0; s < kSegs; ++s) {
            big = max_abs2(max_abs2(big, x[s].x), x[s].y);
            big = max_abs2(max_abs2(big, x[s].z), x[s].w);
            big = max_abs2(max_abs2(big, y[s].x), y[s].y);
            big = max_abs2(max_abs2(big, y[s].z), y[s].w);
        }
        float best0 = -INFINITY, best1 = -INFINITY;
        for (int q0 = 0; q0 < group; q0 += 8) {
            float c[4] = {0.f, 0.f, 0.f, 0.f};
            const uint8_t* qrow = s_q + (q0 + g) * kRowBytes + t * 16;
#pragma unroll
            for (int s = 0; s < kSegs; ++s) {
                const uint4 v = *reinterpret_cast<const uint4*>(qrow + s * 64);
                const uint32_t a0[4] = {x[s].x, y[s].x, x[s].y, y[s].y};
                const uint32_t a1[4] = {x[s].z, y[s].z, x[s].w, y[s].w};
                Mma<T>::run(c, a0, v.x, v.y);
                Mma<T>::run(c, a1, v.z, v.w);
            }
            const bool in0 = q0 + 2 * t < group, in1 = q0 + 2 * t + 1 < group;
            if (in0) best0 = fmaxf(best0, c[0]), best1 = fmaxf(best1, c[2]);
            if (in1) best0 = fmaxf(best0, c[1]), best1 = fmaxf(best1, c[3]);
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            best0 = fmaxf(best0, __shfl_xor_sync(kFull, best0, o));
            best1 = fmaxf(best1, __shfl_xor_sync(kFull, best1, o));
        }
        if (t == 0) {
            float* out = a.scores + unit * a.table_stride + j0;
            if (j0 + g < n) out[g] = use0 ? best0 : -INFINITY;
            if (j0 + g + 8 < n) out[g + 8] = use1 ? best1 : -INFINITY;
        }
    }
    big = max(big & 0xffffu, big >> 16);
    big = __reduce_max_sync(kFull, big);
    if (lane == 0) s_max[warp] = big;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kScoreWarps; ++w) big = max(big, s_max[w]);
        a.tile_max[unit * a.tiles + tile] = big;
    }
}

constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kFew = 256;  // undecided pages that are ranked by comparing all pairs

// Keys whose order as unsigned numbers is that of the scores, NaN above all.
__device__ __forceinline__ uint32_t key_of(float s) {
    if (s != s) return 0xffffffffu;
    const uint32_t u = __float_as_uint(s == 0.f ? 0.f : s);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long key_of(double s) {
    if (s != s) return ~0ull;
    const unsigned long long u = (unsigned long long)__double_as_longlong(s == 0.0 ? 0.0 : s);
    return u >> 63 ? ~u : u | (1ull << 63);
}

// Sum over the CTA, to every thread.  buf: kPickWarps + 1 ints; callers alternate two.
__device__ __forceinline__ int cta_sum(int x, int* buf) {
    x = __reduce_add_sync(kFull, x);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return __reduce_add_sync(kFull, lane < kPickWarps ? buf[lane] : 0);
}

// 64-bit score of a page, worked out by a warp (every lane gets it).
template <typename T, int D>
__device__ __forceinline__ double score64(const SelectArgs& a, int b, int h, int j) {
    const int lane = threadIdx.x & 31;
    const int group = a.n_q_heads / a.n_kv_heads;
    const int page = a.table[(long long)b * a.table_stride + j];
    if (page < 0 || page >= a.num_pages) return -INFINITY;
    const T* row = static_cast<const T*>(a.bounds) + ((long long)page * a.n_kv_heads + h) * 2 * D;
    const T* q = static_cast<const T*>(a.q) + ((long long)b * a.n_q_heads + h * group) * D;
    double best = -INFINITY;
    for (int i = 0; i < group; ++i) {
        double sum = 0.0;
#pragma unroll
        for (int u = 0; u < D / 32; ++u) {
            const int d = u * 32 + lane;
            const float x = (float)q[i * D + d], lo = (float)row[d], hi = (float)row[D + d];
            // as the product does it: both halves, one of them with a zero
            const bool neg = signbit(x);
            sum += (double)(neg ? x : 0.f) * (double)lo + (double)(neg ? 0.f : x) * (double)hi;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        if (sum != sum) return sum;  // every lane has the same sum
        best = fmax(best, sum);
    }
    return best;
}

template <typename T, int D>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const SelectArgs a) {
    __shared__ uint32_t s_chosen[kMaxSelectPages / 32];
    __shared__ int s_buf[2][kPickWarps + 1];
    __shared__ double s_sum[kPickWarps];
    __shared__ uint32_t s_big;
    __shared__ double s_few[kFew];
    __shared__ int s_few_at[kFew];
    __shared__ int s_few_n;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int h = blockIdx.x, b = blockIdx.y;
    const long long unit = (long long)b * a.n_kv_heads + h;
    int32_t* out = a.selected + unit * a.max_pages;
    pdl_wait();
    pdl_trigger();
    uint32_t bits = 0;
    const int n = pages_of(a, b, &bits);  // (flagged by the scores' kernel)
    const int K = a.max_pages;
    if (n <= K) {
        for (int i = threadIdx.x; i < K; i += kPickThreads) out[i] = i < n ? i : -1;
        return;
    }
    // candidates: pages keep_first .. n - keep_last - 1, `want` of them are taken
    const int c0 = a.keep_first, cn = n - a.keep_first - a.keep_last;
    const int want = K - a.keep_first - a.keep_last;
    for (int i = threadIdx.x; i < a.keep_first; i += kPickThreads) out[i] = i;
    for (int i = threadIdx.x; i < a.keep_last; i += kPickThreads)
        out[K - a.keep_last + i] = n - a.keep_last + i;
    if (want == 0) return;
    const float* sc = a.scores + unit * a.table_stride + c0;
    double* sc64 = a.scores64 + unit * a.table_stride + c0;
    const int words = (cn + 31) / 32;
    if (threadIdx.x == 0) {
        s_big = 0;
        s_few_n = 0;
    }
    __syncthreads();

    // S = the largest sum of |q| times the largest |bound|
    {
        const int group = a.n_q_heads / a.n_kv_heads;
        const T* q = static_cast<const T*>(a.q) + ((long long)b * a.n_q_heads + h * group) * D;
        double most = 0.0;
        for (int i = warp; i < group; i += kPickWarps) {
            float sum = 0.f;
#pragma unroll
            for (int u = 0; u < D / 32; ++u) sum += fabsf((float)q[i * D + u * 32 + lane]);
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
            most = sum > most || sum != sum ? (double)sum : most;
        }
        if (lane == 0) s_sum[warp] = most;
        uint32_t big = 0;
        for (int i = threadIdx.x; i < (n + kSelectTile - 1) / kSelectTile; i += kPickThreads)
            big = max(big, a.tile_max[unit * a.tiles + i]);
        big = __reduce_max_sync(kFull, big);
        if (lane == 0) atomicMax(&s_big, big);
    }
    __syncthreads();
    double most = 0.0;
#pragma unroll
    for (int w = 0; w < kPickWarps; ++w) {
        const double x = s_sum[w];
        most = x > most || x != x ? x : most;
    }
    const uint16_t big16 = (uint16_t)s_big;
    const double S = most * (double)(float)(*reinterpret_cast<const T*>(&big16));
    // beyond fp32 (or not a number): no fp32 score says anything
    const bool blind = !(S < 1e38);
    // (2^-126: what a product below fp32's normal range may lose, 256 times)
    const double e2 = 2.0 * (S * 3.0517578125e-05 + (S > 0.0 ? 256.0 * 1.1754943508222875e-38 : 0.0));

    // T: the want-th largest fp32 score, bit by bit from the top
    double upper = INFINITY, lower = -INFINITY;
    int turn = 0;
    if (!blind) {
        uint32_t key = 0;
        for (int bit = 31; bit >= 0; --bit) {
            const uint32_t probe = key | (1u << bit);
            int count = 0;
            for (int i = threadIdx.x; i < cn; i += kPickThreads) count += key_of(sc[i]) >= probe;
            if (cta_sum(count, s_buf[turn ^= 1]) >= want) key = probe;
        }
        const float kth = __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
        upper = (double)kth + e2;
        lower = (double)kth - e2;
        // (e2 infinite cannot be; kth = -inf: bad pages fill up the list, lower = upper = -inf)
    }
    // pages that are chosen for certain, and how many are not settled
    int sure = 0, open = 0;
    for (int w = warp; w < words; w += kPickWarps) {
        const int i = w * 32 + lane;
        const double s = i < cn ? (double)sc[i] : 0.0;
        const bool yes = i < cn && !blind && s > upper;
        const bool may = i < cn && !yes && (blind || s >= lower);
        const uint32_t m = __ballot_sync(kFull, yes);
        if (lane == 0) s_chosen[w] = m;
        sure += yes;
        open += may;
    }
    sure = cta_sum(sure, s_buf[turn ^= 1]);
    open = cta_sum(open, s_buf[turn ^= 1]);
    const int left = want - sure;  // >= 1: at most want - 1 scores are above the want-th
    __syncthreads();

    if (open == left) {  // all of them
        for (int w = warp; w < words; w += kPickWarps) {
            const int i = w * 32 + lane;
            const bool may = i < cn && (blind || ((double)sc[i] >= lower && (double)sc[i] <= upper));
            const uint32_t m = __ballot_sync(kFull, may);
            if (lane == 0) s_chosen[w] |= m;
        }
    } else {
        const bool few = open <= kFew;
        for (int w = warp; w < words; w += kPickWarps) {
            const int i = w * 32 + lane;
            const bool may = i < cn && (blind || ((double)sc[i] >= lower && (double)sc[i] <= upper));
            uint32_t m = __ballot_sync(kFull, may);
            while (m) {
                const int at = w * 32 + __ffs(m) - 1;
                m &= m - 1;
                // S = 0: every product is a zero
                const double s = S == 0.0 ? 0.0 : score64<T, D>(a, b, h, c0 + at);
                if (lane == 0) {
                    if (few) {
                        const int k = atomicAdd(&s_few_n, 1);
                        s_few[k] = s;
                        s_few_at[k] = at;
                    } else {
                        sc64[at] = s;
                    }
                }
            }
        }
        __syncthreads();
        if (few) {
            for (int k = threadIdx.x; k < open; k += kPickThreads) {
                const unsigned long long mine = key_of(s_few[k]);
                const int at = s_few_at[k];
                int above = 0;
                for (int o = 0; o < open; ++o) {
                    const unsigned long long other = key_of(s_few[o]);
                    above += other > mine || (other == mine && s_few_at[o] < at);
                }
                if (above < left) atomicOr(&s_chosen[at >> 5], 1u << (at & 31));
            }
        } else {
            // the left-th largest of the 64-bit scores, bit by bit, then the lowest indexes
            // among its equals
            auto is_open = [&](int i) {
                return blind || ((double)sc[i] >= lower && (double)sc[i] <= upper);
            };
            unsigned long long key = 0;
            for (int bit = 63; bit >= 0; --bit) {
                const unsigned long long probe = key | (1ull << bit);
                int count = 0;
                for (int i = threadIdx.x; i < cn; i += kPickThreads)
                    if (is_open(i)) count += key_of(sc64[i]) >= probe;
                if (cta_sum(count, s_buf[turn ^= 1]) >= left) key = probe;
            }
            int above = 0;
            for (int i = threadIdx.x; i < cn; i += kPickThreads)
                if (is_open(i)) above += key_of(sc64[i]) > key;
            above = cta_sum(above, s_buf[turn ^= 1]);
            int equal = left - above;  // of the equals, the first so many
            for (int w0 = 0; w0 < words; w0 += kPickWarps) {
                const int w = w0 + warp, i = w * 32 + lane;
                const bool may = i < cn && is_open(i);
                const unsigned long long k = may ? key_of(sc64[i]) : 0ull;
                const uint32_t yes = __ballot_sync(kFull, may && k > key);
                uint32_t tie = __ballot_sync(kFull, may && k == key);
                int* buf = s_buf[turn ^= 1];
                if (lane == 0) buf[warp] = __popc(tie);
                __syncthreads();
                int before = 0, all = 0;
#pragma unroll
                for (int x = 0; x < kPickWarps; ++x) {
                    before += x < warp ? buf[x] : 0;
                    all += buf[x];
                }
                int room = equal - before;
                uint32_t take = yes;
                while (tie && room > 0) {
                    take |= tie & -tie;
                    tie &= tie - 1;
                    --room;
                }
                if (lane == 0 && w < words) s_chosen[w] |= take;
                equal -= min(all, max(equal, 0));
            }
        }
    }
    __syncthreads();

    // the chosen in ascending order
    int done = 0;
    for (int w0 = 0; w0 < words; w0 += kPickThreads) {
        const int w = w0 + threadIdx.x;
        uint32_t m = w < words ? s_chosen[w] : 0;
        const int mine = __popc(m);
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(kFull, upto, o);
            if (lane >= o) upto += x;
        }
        int* buf = s_buf[turn ^= 1];
        if (lane == 31) buf[warp] = upto;
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int x = 0; x < kPickWarps; ++x) {
            before += x < warp ? buf[x] : 0;
            all += buf[x];
        }
        int at = done + before + upto - mine;
        while (m) {
            out[c0 + at++] = c0 + w * 32 + __ffs(m) - 1;
            m &= m - 1;
        }
        done += all;
    }
}

template <typename T, int D>
cudaError_t launch(const SelectArgs& a, cudaStream_t stream) {
    const int group = a.n_q_heads / a.n_kv_heads;
    const size_t smem = (size_t)((group + 7) / 8 * 8) * (4 * D + 64);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(
            score_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    cudaError_t e = launch_pdl(score_kernel<T, D>, dim3(a.n_kv_heads, a.tiles, a.batch),
                               dim3(kScoreWarps * 32), smem, stream, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(pick_kernel<T, D>, dim3(a.n_kv_heads, a.batch), dim3(kPickThreads), 0,
                      stream, a);
}

}  // namespace

cudaError_t launch_select(const SelectArgs& a, bool bf16, int head_dim, cudaStream_t stream) {
    if (bf16)
        return head_dim == 128 ? launch<__nv_bfloat16, 128>(a, stream)
                               : launch<__nv_bfloat16, 64>(a, stream);
    return head_dim == 128 ? launch<__half, 128>(a, stream) : launch<__half, 64>(a, stream);
}

}  // namespace pkv
