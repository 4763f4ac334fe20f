// tables.cu -- page tables, slots and positions of a batch's new tokens.
//
// Two exclusive prefix sums over the requests (new tokens, new pages) say where a
// request's token rows start and which entries of the free list are its own; a token
// row i then belongs to the last request that starts at or before i, and its page is
// an old table entry (the partly filled last page) or an entry of the free list.
//
// What bounds it: latency.  The bytes are 16 a token, so a decode step is one dependent
// chain (lengths, sums, page ids, stores).  Every CTA therefore works the sums out for
// itself, in shared memory, rather than wait for another launch that does it once: the
// lengths of 256 requests are 2 KB from L2.  No CTA reads what another one writes
// (a request's old entries are below its new ones), so there is nothing to wait for.
// One scan serves both sums, although a request without token rows takes no pages: the
// requests that have rows all come before the first that has none.  A token a thread: 64
// requests of a token each 2.5 us, 256 requests with 33,500 tokens 3.0 us (four tokens a
// thread and a scan a sum: 6.0).
#include "selected.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Exclusive sums over the CTA of one (tokens, pages) pair a thread; totals in *all_*.
template <typename S>
__device__ __forceinline__ void scan2(S& t, S& g, S* all_t, S* all_g, S (*s_warp)[2]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    S x = t, y = g;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const S a = __shfl_up_sync(kFull, x, o), b = __shfl_up_sync(kFull, y, o);
        if (lane >= o) {
            x += a;
            y += b;
        }
    }
    if (lane == 31) {
        s_warp[warp][0] = x;
        s_warp[warp][1] = y;
    }
    __syncthreads();
    S pt = 0, pg = 0, st = 0, sg = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const S a = s_warp[w][0], b = s_warp[w][1];
        if (w < warp) {
            pt += a;
            pg += b;
        }
        st += a;
        sg += b;
    }
    t = pt + x - t;
    g = pg + y - g;
    *all_t = st;
    *all_g = sg;
}

// S: holds the sums of kThreads requests, each of which counts for at most n_tokens + 1 tokens
// and as many pages.
template <typename S>
__global__ void __launch_bounds__(kThreads) tables_kernel(const TablesArgs a, int per_cta) {
    extern __shared__ int32_t smem[];
    const int B = a.batch, P = a.page_size;
    int32_t* s_start = smem;               // [B + 1] first token row
    int32_t* s_page = smem + B + 1;        // [B] pages taken before the request; -1: refused
    int32_t* s_cached = s_page + B;        // [B]
    __shared__ S s_warp[2][kWarps][2];
    __shared__ uint32_t s_status;
    __shared__ int s_taken;
    if (threadIdx.x == 0) {
        s_status = 0;
        s_taken = 0;
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int begin = a.free_begin ? *a.free_begin : 0;
    int avail = a.n_free - begin;
    uint32_t bits = 0;
    if (begin < 0 || avail < 0) {  // no such entry: nothing is left
        avail = 0;
        bits |= PKV_DEV_NO_PAGES;
    }
    // positions are int32: a request may end at 2^31 - 1 at most
    const long long cap = min((long long)a.table_stride * P, 0x7fffffffLL);

    long long base_t = 0, base_g = 0;
    int turn = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads, turn ^= 1) {
        const int b = b0 + threadIdx.x;
        int c = 0, n = 0;
        if (b < B) {
            c = a.cached[b];
            n = a.fresh[b];
        }
        const bool bad = c < 0 || n < 0;
        c = max(c, 0);
        n = max(n, 0);
        const bool fits_row = !bad && (long long)c + n <= cap;
        // a request that is too long for the rows counts as just too long.  Its pages and
        // those behind it may count or not: no request behind it has rows left
        const int tokens = min(n, a.n_tokens < 0x7fffffff ? a.n_tokens + 1 : a.n_tokens);
        // (c and n fit a row here, whose pages are an int)
        const int need = fits_row ? (int)(((unsigned)c + (unsigned)n + P - 1) / P -
                                          ((unsigned)c + P - 1) / P)
                                  : 0;
        S t = tokens, g = min(need, tokens), all_t, all_g;
        scan2<S>(t, g, &all_t, &all_g, s_warp[turn]);
        const long long start = base_t + (long long)t, end = start + n;
        const long long upto = base_g + (long long)g + need;
        const bool fits = fits_row && end <= a.n_tokens;
        const bool paid = need == 0 || upto <= avail;
        if (b < B) {
            if (!fits) bits |= PKV_DEV_BAD_LEN;
            else if (!paid) bits |= PKV_DEV_NO_PAGES;
            if (fits && paid && need > 0) atomicMax(&s_taken, (int)upto);
            s_start[b] = (int)min(start, (long long)a.n_tokens);
            // (a request that needs no page has no use for the count)
            s_page[b] = fits && paid ? (need ? (int)(upto - need) : 0) : -1;
            s_cached[b] = c;
            if (blockIdx.x == 0) {
                a.lens[b] = fits && paid ? c + n : c;
                a.starts[b] = s_start[b];
            }
        }
        base_t += (long long)all_t;
        base_g += (long long)all_g;
    }
    const int total = (int)min(base_t, (long long)a.n_tokens);
    if (threadIdx.x == 0) s_start[B] = total;
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.starts[B] = total;
        *a.free_end = begin + s_taken;
    }

    // (counted from the CTA's first row: a row's number may be up to 2^31 - 2)
    const long long first = (long long)blockIdx.x * per_cta;
    const int rows = (int)min((long long)per_cta, a.n_tokens - first);
    for (int x = threadIdx.x; x < rows; x += kThreads) {
        const int i = (int)first + x;
        int pos = -1, seq = -1;
        long long slot = -1;
        if (i < total) {
            // the last request with start <= i (empty ones in front of it start there too)
            int lo = 0, hi = B;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (s_start[mid] <= i) lo = mid;
                else hi = mid;
            }
            seq = lo;
            const int pages = s_page[seq];
            if (pages >= 0) {
                const unsigned c = s_cached[seq];
                pos = (int)c + (i - s_start[seq]);
                const int j = pos / P, off = pos - j * P;
                const int have = (int)((c + P - 1) / P);
                int32_t* entry = a.table + (long long)seq * a.table_stride + j;
                int page;
                if (j < have) {
                    page = *entry;
                } else {
                    page = a.free_pages[begin + pages + (j - have)];
                    if (off == 0) *entry = page;  // a new page's first row is a new token's
                }
                if (page < 0 || page >= a.num_pages) bits |= PKV_DEV_BAD_PAGE;
                else slot = (long long)page * P + off;
            }
        }
        a.positions[i] = pos;
        a.seq_ids[i] = seq;
        a.slots[i] = slot;
    }
    if (bits) atomicOr(&s_status, bits);
    __syncthreads();
    if (threadIdx.x == 0 && s_status) set_status(a.status, s_status);
}

}  // namespace

cudaError_t launch_tables(const TablesArgs& a, cudaStream_t stream) {
    // a token a thread while that is a wave of four CTAs an SM, more beyond it
    const long long tiles = a.n_tokens > 0 ? 1 + ((long long)a.n_tokens - 1) / kThreads : 1;
    const long long wave = 4LL * sm_count();
    const int per_cta = (int)((tiles + wave - 1) / wave) * kThreads;
    const int ctas = a.n_tokens > 0 ? (int)(1 + ((long long)a.n_tokens - 1) / per_cta) : 1;
    const size_t smem = (size_t)(3 * a.batch + 1) * 4;
    // sums of kThreads requests in 32 bits
    const bool narrow = a.n_tokens < 0x7fffffff / kThreads - 1;
    auto kernel = narrow ? tables_kernel<int> : tables_kernel<long long>;
    // (the 48 KB that a launch has unasked hold the kernel's static shared memory too)
    static SmemLimit limits[2];
    const cudaError_t e = limits[narrow].set(reinterpret_cast<const void*>(kernel),
                                             (3 * kMaxTableBatch + 1) * 4);
    if (e != cudaSuccess) return e;
    return launch_pdl(kernel, dim3(ctas), dim3(kThreads), smem, stream, a, per_cta);
}

}  // namespace pkv
