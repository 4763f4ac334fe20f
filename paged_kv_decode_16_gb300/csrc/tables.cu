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
#include "selected.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kTokensPerCta = 1024;
constexpr int kWarps = kThreads / 32;

// Exclusive sums over the CTA of one (tokens, pages) pair a thread; totals in *all_*.
__device__ __forceinline__ void scan2(long long& t, long long& g, long long* all_t,
                                      long long* all_g, longlong2* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long x = t, y = g;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long a = __shfl_up_sync(kFull, x, o), b = __shfl_up_sync(kFull, y, o);
        if (lane >= o) {
            x += a;
            y += b;
        }
    }
    if (lane == 31) s_warp[warp] = make_longlong2(x, y);
    __syncthreads();
    long long pt = 0, pg = 0, st = 0, sg = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const longlong2 v = s_warp[w];
        if (w < warp) {
            pt += v.x;
            pg += v.y;
        }
        st += v.x;
        sg += v.y;
    }
    t = pt + x - t;
    g = pg + y - g;
    *all_t = st;
    *all_g = sg;
    __syncthreads();
}

__global__ void __launch_bounds__(kThreads) tables_kernel(const TablesArgs a) {
    extern __shared__ int32_t smem[];
    int32_t* s_start = smem;                 // [B + 1] first token row
    int32_t* s_page = smem + a.batch + 1;    // [B] pages taken before the request; -1: refused
    __shared__ longlong2 s_warp[kWarps];
    __shared__ uint32_t s_status;
    __shared__ int s_taken;
    const int B = a.batch, P = a.page_size;
    if (threadIdx.x == 0) {
        s_status = 0;
        s_taken = 0;
    }
    pdl_wait();
    pdl_trigger();
    int begin = a.free_begin ? *a.free_begin : 0;
    int avail = a.n_free - begin;
    uint32_t bits = 0;
    if (begin < 0 || avail < 0) {  // no such entry: nothing is left
        avail = 0;
        bits |= PKV_DEV_NO_PAGES;
    }
    // positions are int32: a request may end at 2^31 - 1 at most
    const long long cap = min((long long)a.table_stride * P, 0x7fffffffLL);
    __syncthreads();

    long long base_t = 0, base_g = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + threadIdx.x;
        int c = 0, n = 0;
        if (b < B) {
            c = a.cached[b];
            n = a.fresh[b];
        }
        const bool bad = c < 0 || n < 0;
        c = max(c, 0);
        n = max(n, 0);
        const bool fits_row = (long long)c + n <= cap;
        long long t = n, all_t, all_g;
        const long long need_row = ((long long)c + n + P - 1) / P - ((long long)c + P - 1) / P;
        // whether its rows exist depends on the token sum alone: sum that first
        long long g = 0;
        scan2(t, g, &all_t, &all_g, s_warp);
        const long long start = base_t + t, end = start + n;
        const bool fits = !bad && fits_row && end <= a.n_tokens;
        const long long need = fits ? need_row : 0;
        long long none = 0, unused;
        g = need;
        scan2(none, g, &unused, &all_g, s_warp);
        const long long before = base_g + g, upto = before + need;
        const bool paid = need == 0 || upto <= avail;
        if (b < B) {
            if (!fits) bits |= PKV_DEV_BAD_LEN;
            if (!paid) bits |= PKV_DEV_NO_PAGES;
            if (fits && paid && need > 0) atomicMax(&s_taken, (int)upto);
            s_start[b] = (int)min(start, (long long)a.n_tokens);
            // (a request that needs no page has no use for the count)
            s_page[b] = fits && paid ? (need ? (int)before : 0) : -1;
            if (blockIdx.x == 0) {
                a.lens[b] = fits && paid ? c + n : c;
                a.starts[b] = s_start[b];
            }
        }
        base_t += all_t;
        base_g += all_g;
    }
    const int total = (int)min(base_t, (long long)a.n_tokens);
    if (threadIdx.x == 0) s_start[B] = total;
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        a.starts[B] = total;
        *a.free_end = begin + s_taken;
    }

    const int first = blockIdx.x * kTokensPerCta;
    const int last = min(first + kTokensPerCta, a.n_tokens);
    for (int i = first + threadIdx.x; i < last; i += kThreads) {
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
                const int c = a.cached[seq];
                pos = c + (i - s_start[seq]);
                const int j = pos / P, off = pos - j * P;
                const int have = (int)(((long long)c + P - 1) / P);
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
    const int ctas = a.n_tokens > 0 ? 1 + (a.n_tokens - 1) / kTokensPerCta : 1;
    const size_t smem = (size_t)(2 * a.batch + 1) * 4;
    if (smem > 48 * 1024) {
        static SmemLimit limit;
        const cudaError_t e = limit.set(reinterpret_cast<const void*>(tables_kernel),
                                        (2 * kMaxTableBatch + 1) * 4);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(tables_kernel, dim3(ctas), dim3(kThreads), smem, stream, a);
}

}  // namespace pkv
