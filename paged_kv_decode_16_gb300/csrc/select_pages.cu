// select_pages.cu -- the pages that a query attends to: scores, then the choice.
//
// Score of page j for KV head h: max over the head's queries of q+ . hi_j + q- . lo_j, with
// q+ = max(q, 0) and q- = min(q, 0), which is at least q . k for every key of the page.  The
// bounds of a page and head lie as one row [lo | hi] of 2 D elements, so a score is one dot
// product of that row with [q- | q+]: pages are the rows of a matrix product on the
// tensor cores (mma.sync m16n8k16: 16 pages x 8 queries), fed straight from global memory:
// the contraction's order is free, so a lane takes 16 contiguous bytes of a row as its
// fragments of two k-steps.  What bounds it: memory, 4 D bytes a page and head (256 units of
// 8192 pages, 1.07 GB: 187 us with the choice, 5.7 TB/s), and for less the grid's start and
// the choice's phases (256 uneven units of 256 to 2048 pages, 113 MB: 30.4 us, of which 7 the
// choice; 256 units of 64 pages 7.7 us, of which 1.5 where scores near the border are told
// apart).
//
// The choice does not depend on how the product is summed: it tells scores apart to 47 bits of
// the sum of their terms' sizes (long_score).  A product of two 16-bit values is exact in fp32; each of the 2 D / 16 steps adds 16
// of them to the sum, every addend cut at 2^-24 of the largest at worst: 17 addends, 2 D /
// 16 <= 16 steps, so a score is off by at most e = 2^-15 S (S = sum |q_d| max |bound|; the
// count gives 2^-15.9, the last sum of two chains included).  The k-th largest score is then
// off by at most e too: pages more than 2 e above the k-th fp32 score are chosen, those more
// than 2 e below are not, and only the few in between are scored again to more bits, where
// that is not settled by their number.
#include "decode_mma.cuh"
#include "selected.cuh"

namespace pkv {
namespace {

constexpr int kScoreThreads = 128;
constexpr int kPickThreads = 512;
constexpr int kSmallThreads = 256;  // of the kernel that does both
constexpr int kSmallPages = 512;    // and the most table columns it takes
constexpr int kFew = 256;           // pages that are ranked by comparing all pairs
constexpr int kBins = 1024;         // of the histogram that finds the border
// Up to so many candidates are all ranked instead: 60 candidates 4.7 against 5.1 us a call,
// 125 the same, 253 11.1 against 9.4.
constexpr int kRankAll = 64;
constexpr int kScoreCache = 16384;  // scores kept in shared memory
// 2^-60: products that add up to less may have lost, in fp32, last bits that count
constexpr float kSmallSum = 8.673617379884035e-19f;

__device__ __forceinline__ int pages_of(const SelectArgs& a, int b, uint32_t* bits) {
    int len = a.lens[b];
    const long long cap = (long long)a.table_stride * a.page_size;
    if (len < 0 || len > cap) {
        *bits |= PKV_DEV_BAD_LEN;
        len = len < 0 ? 0 : (int)cap;
    }
    return (int)(((long long)len + a.page_size - 1) / a.page_size);
}

// Largest magnitudes of packed 16-bit floats, NaN above all.
template <typename T>
struct Abs2;
template <>
struct Abs2<__nv_bfloat16> {
    using V = __nv_bfloat162;
};
template <>
struct Abs2<__half> {
    using V = __half2;
};
template <typename T>
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t x) {
    using V = typename Abs2<T>::V;
    const V a = __habs2(*reinterpret_cast<const V*>(&x));
    const V r = __hmax2_nan(*reinterpret_cast<const V*>(&m), a);
    return *reinterpret_cast<const uint32_t*>(&r);
}

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

__device__ __forceinline__ float score_of(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key ^ 0x80000000u : ~key);
}

// 16 bytes of a row.  A row is 512 bytes (D 128) somewhere in memory, which its four lanes
// walk 64 bytes at a time: the hint brings 256 into L2 at the first touch (32 requests of
// up to 32768 tokens 33.3 -> 31.5 us a call).
__device__ __forceinline__ uint4 load_row(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// The score of a page for one query head to more than 32 bits, as a key, worked out by D / 8
// lanes side by side (each gets it; page < 0: the key of -inf).  fp64 runs at a 64th of fp32's
// rate on this part, so it serves only where fp32 cannot hold the products: where those of any
// page may be too large (`wide`), or where this page's are too small (for the whole warp then).
// Else a product, exact in fp32, is cut at two bits that go by S, the sum of this page's
// products' sizes, by adding and taking away 1.5 times a power of two: with 2^k above 2 S, the
// parts down to 2^(k-23) add up without rounding, and so do those from there to 2^(k-39); what
// is left is below 2^(k-40), so its rounded sum is off by 2^(k-50), 2^-48 S, at most.
template <typename T, int D>
__device__ __forceinline__ unsigned long long long_score(const SelectArgs& a, int b, int h,
                                                         int page, int head, bool wide) {
    constexpr int kLanes = D / 8;
    const int l = threadIdx.x % kLanes;
    const bool real = page >= 0 && page < a.num_pages;
    const int group = a.n_q_heads / a.n_kv_heads;
    const uint4* row = reinterpret_cast<const uint4*>(
        static_cast<const T*>(a.bounds) + ((long long)page * a.n_kv_heads + h) * 2 * D) + l;
    const uint4* q = reinterpret_cast<const uint4*>(
        static_cast<const T*>(a.q) + ((long long)b * a.n_q_heads + h * group + head) * D) + l;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    double sum = 0.0;
    float p[8], S = 0.f;
    if (!wide) {
        float x[8], lo[8], hi[8];
        Cvt<T>::unpack8(real ? *q : zero, x);
        Cvt<T>::unpack8(real ? *row : zero, lo);
        Cvt<T>::unpack8(real ? row[kLanes] : zero, hi);
        bool some = false;  // a product that is not 0
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float y = signbit(x[e]) ? lo[e] : hi[e];
            p[e] = __fmul_rn(x[e], y);
            S += fabsf(p[e]);
            some = some || (x[e] != 0.f && y != 0.f);
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) S += __shfl_xor_sync(kFull, S, o);
        wide = __any_sync(kFull, some && S < kSmallSum);
        S = fmaxf(S, kSmallSum);
    }
    if (wide) {  // (rare: the rows are read again rather than kept)
        float x[8], lo[8], hi[8];
        Cvt<T>::unpack8(real ? load_row(q) : zero, x);
        Cvt<T>::unpack8(real ? load_row(row) : zero, lo);
        Cvt<T>::unpack8(real ? load_row(row + kLanes) : zero, hi);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // as the product does it: both halves, one of them with a zero
            const bool neg = signbit(x[e]);
            sum += (double)(neg ? x[e] : 0.f) * (double)lo[e];
            sum += (double)(neg ? 0.f : x[e]) * (double)hi[e];
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    } else {
        const uint32_t top = (__float_as_uint(S) >> 23) + 2;  // 2^k: above 2 S
        const float cut1 = __uint_as_float(top << 23 | 0x400000u);
        const float cut2 = __uint_as_float((top - 16) << 23 | 0x400000u);
        float s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float p1 = __fsub_rn(__fadd_rn(p[e], cut1), cut1), r = __fsub_rn(p[e], p1);
            const float p2 = __fsub_rn(__fadd_rn(r, cut2), cut2);
            s1 = __fadd_rn(s1, p1);
            s2 = __fadd_rn(s2, p2);
            s3 = __fadd_rn(s3, __fsub_rn(r, p2));
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) {
            s1 += __shfl_xor_sync(kFull, s1, o);
            s2 += __shfl_xor_sync(kFull, s2, o);
            s3 += __shfl_xor_sync(kFull, s3, o);
        }
        sum = (double)s1 + ((double)s2 + (double)s3);
    }
    return key_of(real ? sum : -(double)INFINITY);
}

// What a tile of scores leaves for the choice.
struct ScoreScratch {
    uint32_t big[16], top[16], low[16];
    float sum[16];
};

// Scores of pages first .. end - 1 of n (by the CTA), and of them the largest |bound|, the keys
// of the largest and the smallest score of a page of the pool, and the largest sum of a
// query's |q|.  The pages that are listed anyway are not read, and have no part in these (what
// they hold must not widen the border of the others).  ids (nullable): receives the pages
// (-1: not one of the pool's, or listed anyway).
template <typename T, int D, int THREADS>
__device__ __forceinline__ void score_pages(const SelectArgs& a, int b, int h, int first, int end,
                                            int n, uint8_t* s_q, ScoreScratch& sh, uint4* stat,
                                            int* ids = nullptr) {
    constexpr int kSegs = 2 * D / 32;      // 64-byte pieces of a row: two k-steps each
    constexpr int kRowBytes = 4 * D + 64;  // a query's [q- | q+], rows 64 bytes apart mod 128
    constexpr int kWarps = THREADS / 32, kStep = kWarps * 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = a.n_q_heads / a.n_kv_heads;
    const int rows8 = (group + 7) / 8 * 8;
    const int32_t* table = a.table + (long long)b * a.table_stride;
    const T* bounds = static_cast<const T*>(a.bounds) + (long long)h * 2 * D;
    const long long page_step = (long long)a.n_kv_heads * 2 * D;
    const int g = lane >> 2, t = lane & 3;
    uint32_t bits = 0;
    // lanes 0 .. 15 (and again 16 .. 31) find the pages, every lane then takes rows g, g + 8
    auto page_at = [&](int j0) {
        const int j = j0 + (lane & 15);
        if (j >= end) return -1;
        int page = table[j];
        if (page < 0 || page >= a.num_pages) {
            bits |= PKV_DEV_BAD_PAGE;
            page = -1;
        }
        if (j < a.keep_first || j >= n - a.keep_last) page = -1;
        if (ids && lane < 16) ids[j] = page;
        return page;
    };
    uint4 x[kSegs], y[kSegs];
    bool use0, use1;
    auto load = [&](int page) {
        const int page0 = __shfl_sync(kFull, page, g), page1 = __shfl_sync(kFull, page, g + 8);
        use0 = page0 >= 0, use1 = page1 >= 0;
        const uint4* r0 = reinterpret_cast<const uint4*>(bounds + page0 * page_step);
        const uint4* r1 = reinterpret_cast<const uint4*>(bounds + page1 * page_step);
#pragma unroll
        for (int s = 0; s < kSegs; ++s) {
            x[s] = y[s] = make_uint4(0, 0, 0, 0);
            if (use0) x[s] = load_row(r0 + s * 4 + t);
            if (use1) y[s] = load_row(r1 + s * 4 + t);
        }
    };
    int j0 = first + warp * 16;
    load(page_at(j0));  // in flight while the queries come
    int next = page_at(j0 + kStep);

    // [q- | q+] of the head's queries; rows behind the group are zeros and not used
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) +
                                                    ((long long)b * a.n_q_heads + h * group) * D);
    for (int i = threadIdx.x; i < rows8 * (D / 8); i += THREADS) {
        const int r = i / (D / 8), c = i % (D / 8);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (r < group) v = q[i];
        uint32_t w[4] = {v.x, v.y, v.z, v.w}, neg[4], pos[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // by the sign bit; a NaN goes to one of the two and makes the score NaN
            const uint32_t mask = ((w[e] & 0x80008000u) >> 15) * 0xffffu;
            neg[e] = w[e] & mask;
            pos[e] = w[e] & ~mask;
        }
        uint8_t* at = s_q + r * kRowBytes + c * 16;
        *reinterpret_cast<uint4*>(at) = make_uint4(neg[0], neg[1], neg[2], neg[3]);
        *reinterpret_cast<uint4*>(at + 2 * D) = make_uint4(pos[0], pos[1], pos[2], pos[3]);
    }
    __syncthreads();

    const long long unit = (long long)b * a.n_kv_heads + h;
    uint32_t big = 0, top = 0, low = 0xffffffffu;
    for (; j0 < end; j0 += kStep) {
#pragma unroll
        for (int s = 0; s < kSegs; ++s) {
            big = max_abs2<T>(max_abs2<T>(big, x[s].x), x[s].y);
            big = max_abs2<T>(max_abs2<T>(big, x[s].z), x[s].w);
            big = max_abs2<T>(max_abs2<T>(big, y[s].x), y[s].y);
            big = max_abs2<T>(max_abs2<T>(big, y[s].z), y[s].w);
        }
        float best0 = -INFINITY, best1 = -INFINITY;
        for (int q0 = 0; q0 < group; q0 += 8) {
            float c[2][4] = {};  // even and odd k-steps in chains of their own
            const uint8_t* qrow = s_q + (q0 + g) * kRowBytes + t * 16;
#pragma unroll
            for (int s = 0; s < kSegs; ++s) {
                const uint4 v = *reinterpret_cast<const uint4*>(qrow + s * 64);
                const uint32_t a0[4] = {x[s].x, y[s].x, x[s].y, y[s].y};
                const uint32_t a1[4] = {x[s].z, y[s].z, x[s].w, y[s].w};
                Mma<T>::run(c[0], a0, v.x, v.y);
                Mma<T>::run(c[1], a1, v.z, v.w);
            }
            if (q0 + 2 * t < group) {
                best0 = fmaxf(best0, c[0][0] + c[1][0]);
                best1 = fmaxf(best1, c[0][2] + c[1][2]);
            }
            if (q0 + 2 * t + 1 < group) {
                best0 = fmaxf(best0, c[0][1] + c[1][1]);
                best1 = fmaxf(best1, c[0][3] + c[1][3]);
            }
        }
        const bool in0 = use0, in1 = use1;
        if (j0 + kStep < end) {
            load(next);
            next = page_at(j0 + 2 * kStep);
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            best0 = fmaxf(best0, __shfl_xor_sync(kFull, best0, o));
            best1 = fmaxf(best1, __shfl_xor_sync(kFull, best1, o));
        }
        if (t == 0) {
            float* out = a.scores + unit * a.table_stride + j0;
            if (j0 + g < end) out[g] = in0 ? best0 : -INFINITY;
            if (j0 + g + 8 < end) out[g + 8] = in1 ? best1 : -INFINITY;
            if (in0) top = max(top, key_of(best0)), low = min(low, key_of(best0));
            if (in1) top = max(top, key_of(best1)), low = min(low, key_of(best1));
        }
    }
    if (bits) set_status(a.status, bits);
    // the sums of |q|: [q- | q+] holds each element once, beside a zero
    float most = 0.f;
    for (int r = warp; r < group; r += kWarps) {
        const uint4* row = reinterpret_cast<const uint4*>(s_q + r * kRowBytes);
        float sum = 0.f;
        if (lane < D / 4) {
            float f[8];
            Cvt<T>::unpack8(row[lane], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += fabsf(f[e]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
        most = sum > most || sum != sum ? sum : most;
    }
    big = __reduce_max_sync(kFull, max(big & 0xffffu, big >> 16));
    top = __reduce_max_sync(kFull, top);
    low = __reduce_min_sync(kFull, low);
    if (lane == 0) {
        sh.big[warp] = big;
        sh.top[warp] = top;
        sh.low[warp] = low;
        sh.sum[warp] = most;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            big = max(big, sh.big[w]);
            top = max(top, sh.top[w]);
            low = min(low, sh.low[w]);
            most = sh.sum[w] > most || sh.sum[w] != sh.sum[w] ? sh.sum[w] : most;
        }
        *stat = make_uint4(big, top, low, __float_as_uint(most));
    }
}

// Sum over the CTA, to every thread.  buf: an int a warp; callers alternate two.
template <int THREADS>
__device__ __forceinline__ int cta_sum(int x, int* buf) {
    x = __reduce_add_sync(kFull, x);
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = x;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    return __reduce_add_sync(kFull, lane < THREADS / 32 ? buf[lane] : 0);
}

struct PickScratch {
    uint32_t chosen[kMaxSelectPages / 32];
    int hist[kBins];
    int buf[2][16];
    int few_at[kFew];              // pages that are not settled, the keys of their scores,
    uint32_t few[kFew];
    unsigned long long far[kFew];  // and of their 64-bit scores
    int open_n, bin;
    uint32_t kth;
};

// The want-th largest of `key_at(i)` over i < cn, bit by bit from the top (any number of
// candidates and equals).
template <int THREADS, typename K, typename F>
__device__ __forceinline__ K kth_key(int (*buf)[16], int& turn, int cn, int want, F key_at) {
    K key = 0;
    for (int bit = 8 * sizeof(K) - 1; bit >= 0; --bit) {
        const K probe = key | ((K)1 << bit);
        int count = 0;
        for (int i = threadIdx.x; i < cn; i += THREADS) count += key_at(i) >= probe;
        if (cta_sum<THREADS>(count, buf[turn ^= 1]) >= want) key = probe;
    }
    return key;
}

// The choice among pages c0 .. c0 + cn - 1: the `want` of the highest scores, into out[c0 ..].
// stats: the unit's tiles'.  ids (nullable): the unit's pages.  sh.hist and sh.open_n are 0.
template <typename T, int D, int THREADS>
__device__ __forceinline__ void pick(const SelectArgs& a, int b, int h, int c0, int cn, int want,
                                     int32_t* out, const uint4* stats, int tiles, float* s_sc,
                                     int cache, PickScratch& sh, const int* ids = nullptr) {
    constexpr int kWarps = THREADS / 32;
    constexpr int kLanes = D / 8, kTeams = 32 / kLanes;  // of a long score
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = a.n_q_heads / a.n_kv_heads;
    const long long unit = (long long)b * a.n_kv_heads + h;
    const float* far = a.scores + unit * a.table_stride + c0;
    unsigned long long* keys64 = a.keys64 + unit * a.table_stride + c0;
    const int words = (cn + 31) / 32;
    int turn = 0;

    for (int i = threadIdx.x; i < min(cn, cache); i += THREADS) s_sc[i] = far[i];
    uint32_t big = 0, top = 0, low = 0xffffffffu;
    float most = 0.f;
    for (int i = lane; i < tiles; i += 32) {
        const uint4 st = stats[i];
        big = max(big, st.x);
        top = max(top, st.y);
        low = min(low, st.z);
        most = __uint_as_float(st.w);  // the same for every tile
    }
    big = __reduce_max_sync(kFull, big);
    top = __reduce_max_sync(kFull, top);
    low = __reduce_min_sync(kFull, low);
    most = __shfl_sync(kFull, most, 0);
    const uint16_t big16 = (uint16_t)big;
    // S and twice the error bound, rounded up
    const float S = __fmul_ru(most, (float)(*reinterpret_cast<const T*>(&big16)));
    // beyond fp32 (or not a number): no fp32 score says anything
    const bool blind = !(S < 1e36f);
    // (the second part: what products below fp32's normal range may lose, 256 of them, twice)
    const float e2 = S > 0.f ? __fadd_ru(__fmul_ru(S, 6.103515625e-05f), 6.1e-36f) : 0.f;
    const int team = lane / kLanes;
    auto page_of = [&](int i) {
        return ids ? ids[c0 + i] : a.table[(long long)b * a.table_stride + c0 + i];
    };
    auto score = [&](int i) { return i < cache ? s_sc[i] : far[i]; };

    // Where the border lies: for few candidates by their ranks; else the want-th largest fp32
    // score is in the bin that the counts reach it in.  (A bin's number grows with the score,
    // whatever the rounding.  A page outside the pool, -inf, falls into bin 0.)
    float upper = INFINITY, lower = -INFINITY;  // above / below is settled
    const float mx = score_of(top), mn = low > top ? mx : score_of(low);
    const float inv = top != 0 && mx > mn ? (float)(kBins - 1) / (mx - mn) : 0.f;
    auto bin_of = [&](float s) { return min(max((int)((s - mn) * inv), 0), kBins - 1); };
    const bool ranked = cn <= kRankAll && cn <= cache;
    if (!blind && ranked) {
        static_assert(kRankAll <= THREADS, "a candidate a thread");
        if (threadIdx.x < 4 && cn + threadIdx.x < (cn + 3) / 4 * 4)
            s_sc[cn + threadIdx.x] = -INFINITY;  // (room for them behind the cache)
        __syncthreads();
        if (threadIdx.x < cn) {
            const float s = s_sc[threadIdx.x];
            int more = 0, up = 0;  // above it; not below it
            for (int j = 0; j < cn; j += 4) {
                const float4 o = *reinterpret_cast<const float4*>(s_sc + j);
                more += (o.x > s) + (o.y > s) + (o.z > s) + (o.w > s);
                up += (o.x >= s) + (o.y >= s) + (o.z >= s) + (o.w >= s);
            }
            // (-inf itself counts the padding too, which lies behind all candidates)
            if (more < want && want <= up) sh.kth = key_of(s);
        }
        __syncthreads();
        const float kth = score_of(sh.kth);
        upper = __fadd_ru(kth, e2);
        lower = __fadd_rd(kth, -e2);
    } else if (!blind) {
        for (int i = threadIdx.x; i < cn; i += THREADS)  // (the thread's own copies)
            atomicAdd(&sh.hist[bin_of(score(i))], 1);
        __syncthreads();
        constexpr int kPer = kBins / THREADS;
        int own[kPer], mine = 0;
#pragma unroll
        for (int e = 0; e < kPer; ++e)
            mine += own[e] = sh.hist[kBins - 1 - (threadIdx.x * kPer + e)];
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, upto, o);
            if (lane >= o) upto += v;
        }
        int* buf = sh.buf[turn ^= 1];
        if (lane == 31) buf[warp] = upto;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) upto += w < warp ? buf[w] : 0;
        int above = upto - mine;
        if (above < want && want <= upto) {  // one thread
#pragma unroll
            for (int e = 0; e < kPer; ++e) {
                if (above < want && want <= above + own[e])
                    sh.bin = kBins - 1 - (threadIdx.x * kPer + e);
                above += own[e];
            }
        }
        __syncthreads();
        const int bin = sh.bin;
        // all that may be within 2 e of a score of that bin: the bin's ends (a few roundings
        // of their size further apart) and e2.  One bin for all (inv = 0) has no ends.
        const float slack = __fadd_ru(e2, fmaxf(fabsf(mn), fabsf(mx)) * 2e-6f);
        if (inv > 0.f && bin < kBins - 1) upper = mn + (float)(bin + 1) * (1.0f / inv) + slack;
        if (inv > 0.f && bin > 0) lower = mn + (float)bin * (1.0f / inv) - slack;
    }
    // pages that are chosen for certain, and those that are not settled
    int sure = 0;
    for (int w = warp; w < words; w += kWarps) {
        const int i = w * 32 + lane;
        const float s = i < cn ? score(i) : 0.f;
        const bool yes = i < cn && !blind && s > upper;
        const bool may = i < cn && !yes && (blind || s >= lower);
        const uint32_t m = __ballot_sync(kFull, yes);
        if (lane == 0) sh.chosen[w] = m;
        sure += __popc(m);
        if (may) {
            const int k = atomicAdd(&sh.open_n, 1);
            if (k < kFew) {
                sh.few_at[k] = i;
                sh.few[k] = key_of(s);
                sh.far[k] = 0ull;
            }
        }
    }
    sure = cta_sum<THREADS>(lane == 0 ? sure : 0, sh.buf[turn ^= 1]);
    const int open = sh.open_n;
    int left = want - sure;  // >= 1
    if (open <= kFew && open == left) {  // all of them
        for (int k = threadIdx.x; k < open; k += THREADS)
            atomicOr(&sh.chosen[sh.few_at[k] >> 5], 1u << (sh.few_at[k] & 31));
    } else if (open <= kFew && !blind) {
        bool told = false;
        if (!ranked) {
            // the left-th of the few by fp32: those more than e2 from it are settled too
            for (int k = threadIdx.x; k < open; k += THREADS) {
                const uint32_t s = sh.few[k];
                int more = 0, same = 0;
                for (int o = 0; o < open; ++o) {
                    more += sh.few[o] > s;
                    same += sh.few[o] == s;
                }
                if (more < left && left <= more + same) sh.kth = s;
            }
            __syncthreads();
            const float kth = score_of(sh.kth);
            upper = __fadd_ru(kth, e2);
            lower = __fadd_rd(kth, -e2);
            int yes = 0, may = 0;
            for (int k = lane; k < open; k += 32) {  // every warp counts for itself
                const float s = score_of(sh.few[k]);
                yes += s > upper;
                may += s <= upper && s >= lower;
            }
            yes = __reduce_add_sync(kFull, yes);
            may = __reduce_add_sync(kFull, may);
            told = may == left - yes;
            for (int k = threadIdx.x; k < open; k += THREADS) {
                const float s = score_of(sh.few[k]);
                if (told && s >= lower)
                    atomicOr(&sh.chosen[sh.few_at[k] >> 5], 1u << (sh.few_at[k] & 31));
                if (s > upper) sh.far[k] = ~0ull;  // settled: the end of the keys' range
            }
            __syncthreads();
        }
        if (!told) {
            // the others' 64-bit keys, a team of lanes a (page, head)
            for (int x0 = warp * kTeams; x0 < open * group; x0 += kWarps * kTeams) {
                const int x = x0 + team, k = min(x / group, open - 1);
                const float s = score_of(sh.few[k]);
                const bool mine = x < open * group && s <= upper && s >= lower;
                const int page = mine ? page_of(sh.few_at[k]) : -1;
                const unsigned long long key =
                    long_score<T, D>(a, b, h, page, x - k * group, blind);
                if (mine && lane % kLanes == 0) atomicMax(&sh.far[k], key);
            }
            __syncthreads();
            for (int k = threadIdx.x; k < open; k += THREADS) {
                const unsigned long long mine = sh.far[k];
                const int at = sh.few_at[k];
                int above = 0;
                for (int o = 0; o < open; ++o) {
                    const unsigned long long other = sh.far[o];
                    above += other > mine || (other == mine && sh.few_at[o] < at);
                }
                if (above < left) atomicOr(&sh.chosen[at >> 5], 1u << (at & 31));
            }
        }
    } else {
        // many (scores that crowd into a bin, equal pages, or scores beyond fp32): the
        // exact border of the fp32 scores bit by bit, the 64-bit scores around it into the
        // workspace, the left-th largest of those, then the lowest indexes among its equals
        if (!blind) {
            const float kth = score_of(kth_key<THREADS, uint32_t>(
                sh.buf, turn, cn, want, [&](int i) { return key_of(score(i)); }));
            upper = __fadd_ru(kth, e2);
            lower = __fadd_rd(kth, -e2);
        }
        auto is_open = [&](int i) {
            const float s = score(i);
            return blind || (s >= lower && s <= upper);
        };
        // (S = 0, a query or bounds of zeros: what is open is all equal)
        auto long_key = [&](int i) { return S != 0.f ? keys64[i] : 1ull; };
        sure = 0;
        for (int w = warp; w < words; w += kWarps) {
            const int i = w * 32 + lane;
            const uint32_t yes = __ballot_sync(kFull, i < cn && !blind && score(i) > upper);
            if (lane == 0) sh.chosen[w] = yes;
            sure += __popc(yes);
            uint32_t m = __ballot_sync(kFull, i < cn && is_open(i));
            while (m && S != 0.f) {
                const int at = w * 32 + __ffs(m) - 1;
                m &= m - 1;
                const int page = page_of(at);
                unsigned long long key = 0;
                for (int x = 0; x < group; x += kTeams)  // (the last head again for idle teams)
                    key = max(key,
                              long_score<T, D>(a, b, h, page, min(x + team, group - 1), blind));
#pragma unroll
                for (int o = kLanes; o < 32; o <<= 1)
                    key = max(key, __shfl_xor_sync(kFull, key, o));
                if (lane == 0) keys64[at] = key;
            }
        }
        left = want - cta_sum<THREADS>(lane == 0 ? sure : 0, sh.buf[turn ^= 1]);
        const unsigned long long key = kth_key<THREADS, unsigned long long>(
            sh.buf, turn, cn, left, [&](int i) { return is_open(i) ? long_key(i) : 0ull; });
        int above = 0;
        for (int i = threadIdx.x; i < cn; i += THREADS) above += is_open(i) && long_key(i) > key;
        int equal = left - cta_sum<THREADS>(above, sh.buf[turn ^= 1]);  // the first so many
        for (int w0 = 0; w0 < words; w0 += kWarps) {
            const int w = w0 + warp, i = w * 32 + lane;
            const bool may = i < cn && is_open(i);
            const unsigned long long k = may ? long_key(i) : 0ull;
            uint32_t take = __ballot_sync(kFull, may && k > key);
            uint32_t tie = __ballot_sync(kFull, may && k == key);
            int* buf = sh.buf[turn ^= 1];
            if (lane == 0) buf[warp] = __popc(tie);
            __syncthreads();
            int before = 0, all = 0;
#pragma unroll
            for (int v = 0; v < kWarps; ++v) {
                before += v < warp ? buf[v] : 0;
                all += buf[v];
            }
            for (int room = equal - before; tie && room > 0; --room) {
                take |= tie & -tie;
                tie &= tie - 1;
            }
            if (lane == 0 && w < words) sh.chosen[w] |= take;
            equal -= min(all, max(equal, 0));
        }
    }
    __syncthreads();

    // the chosen in ascending order
    int done = 0;
    for (int w0 = 0; w0 < words; w0 += THREADS) {
        const int w = w0 + threadIdx.x;
        uint32_t m = w < words ? sh.chosen[w] : 0;
        const int mine = __popc(m);
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kFull, upto, o);
            if (lane >= o) upto += v;
        }
        int* buf = sh.buf[turn ^= 1];
        if (lane == 31) buf[warp] = upto;
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int v = 0; v < kWarps; ++v) {
            before += v < warp ? buf[v] : 0;
            all += buf[v];
        }
        int at = done + before + upto - mine;
        while (m) {
            out[c0 + at++] = c0 + w * 32 + __ffs(m) - 1;
            m &= m - 1;
        }
        done += all;
    }
}

// What needs no scores: every page where there are no more than max_pages, and the pages that
// are always kept.  True where nothing is left to choose.
__device__ __forceinline__ bool list_kept(const SelectArgs& a, int n, int32_t* out, int threads,
                                          bool write) {
    const int K = a.max_pages;
    if (n <= K) {  // (K may be close to 2^31: 32 bits without a sign hold the loop's last sum)
        for (uint32_t i = threadIdx.x; write && i < (uint32_t)K; i += threads)
            out[i] = i < (uint32_t)n ? (int)i : -1;
        return true;
    }
    for (int i = threadIdx.x; write && i < a.keep_first; i += threads) out[i] = i;
    for (int i = threadIdx.x; write && i < a.keep_last; i += threads)
        out[K - a.keep_last + i] = n - a.keep_last + i;
    return a.keep_first + a.keep_last == K;
}

template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads) score_kernel(const SelectArgs a) {
    extern __shared__ __align__(16) uint8_t s_q[];
    __shared__ ScoreScratch sh;
    const int h = blockIdx.x, tile = blockIdx.y, b = blockIdx.z;
    pdl_wait();
    pdl_trigger();
    uint32_t bits = 0;
    const int n = pages_of(a, b, &bits);
    if (bits && h == 0 && tile == 0 && threadIdx.x == 0) set_status(a.status, bits);
    const int first = tile * a.tile_pages;
    if (first >= n || list_kept(a, n, nullptr, kScoreThreads, false)) return;
    score_pages<T, D, kScoreThreads>(a, b, h, first, min(first + a.tile_pages, n), n, s_q, sh,
                                     a.stats + ((long long)b * a.n_kv_heads + h) * a.tiles + tile);
}

template <typename T, int D>
__global__ void __launch_bounds__(kPickThreads) pick_kernel(const SelectArgs a, int cache) {
    extern __shared__ __align__(16) float s_sc[];  // [cache + 4]
    __shared__ PickScratch sh;
    const int h = blockIdx.x, b = blockIdx.y;
    const long long unit = (long long)b * a.n_kv_heads + h;
    int32_t* out = a.selected + unit * a.max_pages;
    for (int i = threadIdx.x; i < kBins; i += kPickThreads) sh.hist[i] = 0;
    if (threadIdx.x == 0) sh.open_n = 0;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    uint32_t bits = 0;
    const int n = pages_of(a, b, &bits);  // (flagged by the scores' kernel)
    if (list_kept(a, n, out, kPickThreads, true)) return;
    pick<T, D, kPickThreads>(a, b, h, a.keep_first, n - a.keep_first - a.keep_last,
                             a.max_pages - a.keep_first - a.keep_last, out,
                             a.stats + unit * a.tiles, (n + a.tile_pages - 1) / a.tile_pages, s_sc,
                             cache, sh);
}

// Both in one CTA.
template <typename T, int D>
__global__ void __launch_bounds__(kSmallThreads) select_small_kernel(const SelectArgs a, int cache,
                                                                     int q_bytes) {
    extern __shared__ __align__(16) uint8_t s_dyn[];
    __shared__ ScoreScratch score_sh;
    __shared__ PickScratch sh;
    __shared__ int s_ids[kSmallPages];
    const int h = blockIdx.x, b = blockIdx.y;
    const long long unit = (long long)b * a.n_kv_heads + h;
    int32_t* out = a.selected + unit * a.max_pages;
    for (int i = threadIdx.x; i < kBins; i += kSmallThreads) sh.hist[i] = 0;
    if (threadIdx.x == 0) sh.open_n = 0;
    pdl_wait();
    pdl_trigger();
    uint32_t bits = 0;
    const int n = pages_of(a, b, &bits);
    if (bits && h == 0 && threadIdx.x == 0) set_status(a.status, bits);
    if (list_kept(a, n, out, kSmallThreads, true)) return;
    uint4* stat = a.stats + unit * a.tiles;
    score_pages<T, D, kSmallThreads>(a, b, h, 0, n, n, s_dyn, score_sh, stat, s_ids);
    __syncthreads();
    pick<T, D, kSmallThreads>(a, b, h, a.keep_first, n - a.keep_first - a.keep_last,
                              a.max_pages - a.keep_first - a.keep_last, out, stat, 1,
                              reinterpret_cast<float*>(s_dyn + q_bytes), cache, sh, s_ids);
}

template <typename T, int D>
cudaError_t launch(SelectArgs a, cudaStream_t stream) {
    const int group = a.n_q_heads / a.n_kv_heads;
    const int q_bytes = (group + 7) / 8 * 8 * (4 * D + 64);
    const int cache = a.table_stride < kScoreCache ? a.table_stride : kScoreCache;
    const int cache_bytes = cache * 4 + 16;
    const long long units = (long long)a.batch * a.n_kv_heads;
    // Short rows: one launch, a CTA a unit.  us a call (bf16, D 128), one / two launches, as
    // both were measured: 32 units of 128 pages 8.0 / 9.5, 256 pages 9.3 / 9.9, 512 pages
    // 12.1 / 10.1; 128 units of 512 pages 12.5 / 14.9.  Longer rows of unequal requests want
    // their pages shared out.
    if (a.table_stride <= 256 || (a.table_stride <= kSmallPages && 2 * units >= sm_count())) {
        a.tiles = 1;
        static SmemLimit limit;
        const cudaError_t e = limit.set(reinterpret_cast<const void*>(select_small_kernel<T, D>),
                                        kMaxSelectGroup * (4 * D + 64) + kScoreCache * 4 + 16);
        if (e != cudaSuccess) return e;
        return launch_pdl(select_small_kernel<T, D>, dim3(a.n_kv_heads, a.batch),
                          dim3(kSmallThreads), q_bytes + cache_bytes, stream, a, cache, q_bytes);
    }
    // a few steps a CTA (its start is a chain of loads: length, table, bounds), as long as
    // the CTAs make a wave
    a.tile_pages = kSelectTile;
    const long long wave = 4LL * sm_count();
    while (a.tile_pages < 16 * kSelectTile &&
           units * ((a.table_stride + 2 * a.tile_pages - 1) / (2 * a.tile_pages)) >= wave)
        a.tile_pages *= 2;
    a.tiles = (a.table_stride + a.tile_pages - 1) / a.tile_pages;
    static SmemLimit score_limit, pick_limit;
    cudaError_t e = score_limit.set(reinterpret_cast<const void*>(score_kernel<T, D>),
                                    kMaxSelectGroup * (4 * D + 64));
    if (e == cudaSuccess)
        e = pick_limit.set(reinterpret_cast<const void*>(pick_kernel<T, D>),
                           kScoreCache * 4 + 16);
    if (e == cudaSuccess)
        e = launch_pdl(score_kernel<T, D>, dim3(a.n_kv_heads, a.tiles, a.batch),
                       dim3(kScoreThreads), q_bytes, stream, a);
    if (e != cudaSuccess) return e;
    return launch_pdl(pick_kernel<T, D>, dim3(a.n_kv_heads, a.batch), dim3(kPickThreads),
                      cache_bytes, stream, a, cache);
}

}  // namespace

cudaError_t launch_select(const SelectArgs& a, bool bf16, int head_dim, cudaStream_t stream) {
    if (bf16)
        return head_dim == 128 ? launch<__nv_bfloat16, 128>(a, stream)
                               : launch<__nv_bfloat16, 64>(a, stream);
    return head_dim == 128 ? launch<__half, 128>(a, stream) : launch<__half, 64>(a, stream);
}

}  // namespace pkv
