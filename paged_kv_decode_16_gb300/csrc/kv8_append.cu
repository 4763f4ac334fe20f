// kv8_append.cu -- appending keys and values to the 8-bit paged cache, with
// the optional norm and rotation of q and k in the same pass.
//
// A run is the longest stretch of consecutive tokens of one sequence, at
// consecutive positions, within one block of 16: the unit that sets a block's
// scale.  Its first token (its leader) is found from the token and the one
// before it alone, so a CTA needs no list of sequences: CTA i owns the runs
// whose leaders lie among tokens S i .. S i + S - 1, which are the tokens from
// its first leader up to the next CTA's.  The cos / sin of those tokens are
// formed once in shared memory for all heads; then a group of lanes takes a
// row of q, and a warp takes one (run, head, side): the whole block in
// registers, one pass over the data.
//
// What bounds it: long prompts, HBM (q read and written in 16 bits, K and V
// read in 16 and written in 8); a step's single tokens, latency.
#include <math.h>

#include "kv8.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxSpan = 16 + kChunk - 1;  // tokens a CTA may own (S <= 16)

template <typename T>
__device__ __forceinline__ void unpack(const uint4& v, float (&f)[8]) {
    Cvt<T>::unpack8(v, f);
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[8]) {
    return make_uint4(Cvt<T>::pack2(f[0], f[1]), Cvt<T>::pack2(f[2], f[3]),
                      Cvt<T>::pack2(f[4], f[5]), Cvt<T>::pack2(f[6], f[7]));
}

// cos and sin of position * theta^(-2i/D), from the frequency in turns as a
// 64-bit binary fraction: the product wraps modulo one turn by itself, exactly
// (fp64 products would cost more on this part and lose low bits at far
// positions).  The top 32 bits as a signed fraction of half a turn give the
// angle to 2^-32 turns before its rounding to fp32.
__device__ __forceinline__ void turn_cos_sin(int pos, uint64_t turns, float* c, float* s) {
    const uint64_t ph = (uint64_t)(int64_t)pos * turns;
    const float x = (float)(int)(ph >> 32) * 4.6566128730773926e-10f;  // 2^-31: half turns
    sincospif(x, s, c);
}

// 1 / rms of the row whose elements HV neighbouring lanes hold.
template <int D>
__device__ __forceinline__ float inv_rms(const float (&lo)[8], const float (&hi)[8], float eps) {
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(lo[e], lo[e], fmaf(hi[e], hi[e], sum));
#pragma unroll
    for (int o = D / 32; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    return 1.0f / sqrtf(sum / (float)D + eps);
}

// Norm (wlo non-null: weights of the 8 low and 8 high elements; inv: 1 / rms)
// and rotation (c non-null) of a lane's elements lo[e] and their partners hi[e].
__device__ __forceinline__ void norm_rotate(float (&lo)[8], float (&hi)[8], const float* wlo,
                                            const float* whi, float inv, const float* c,
                                            const float* s) {
    if (wlo) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            lo[e] = lo[e] * inv * wlo[e];
            hi[e] = hi[e] * inv * whi[e];
        }
    }
    if (c) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float a = lo[e], b = hi[e];
            lo[e] = fmaf(a, c[e], -b * s[e]);
            hi[e] = fmaf(b, c[e], a * s[e]);
        }
    }
}

// Eight elements times inv (2^-e) as e4m3 bytes; bad: some element is not
// finite (stored as NaN).
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], float inv, bool bad) {
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        y[e] = x[e] * inv;
        if (bad && !(fabsf(x[e]) <= 3.402823466e38f)) y[e] = __uint_as_float(0x7fc00000u);
    }
    return make_uint2(f2_to_e4m3x2(y[0], y[1]) | f2_to_e4m3x2(y[2], y[3]) << 16,
                      f2_to_e4m3x2(y[4], y[5]) | f2_to_e4m3x2(y[6], y[7]) << 16);
}

struct Run {
    int tok;   // its first token
    int n;     // tokens
    int lo;    // slot of the first token in its block
    long long blk;  // block of the pool at head 0: page * Hkv * (P / 16) + block of the page
};

// One (run, head, side) by a warp.  The rows stay packed in registers; what is
// computed from them (the norm, the rotation) is computed twice, for the largest
// element and for the bytes, which costs less than the registers for it would in
// warps at work (64 more a thread).
template <typename T, int D, bool kK>
__device__ __forceinline__ void append_block(const Kv8AppendArgs& a, const Run& r, int h,
                                             int tok0, const float* ctab, const float* stab,
                                             const float* wk, int lane) {
    constexpr int HV = D / 16;        // lanes a row
    constexpr int RPP = 32 / HV;      // rows a pass
    constexpr int PASSES = kChunk / RPP;
    const int jl = lane % HV, rl = lane / HV;
    const uint4* src = static_cast<const uint4*>(kK ? a.k_new : a.v_new);
    uint4 vl[PASSES], vh[PASSES];
    float inv[PASSES];
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
        const int x = ps * RPP + rl;  // token of the run
        vl[ps] = vh[ps] = make_uint4(0u, 0u, 0u, 0u);
        if (x < r.n) {
            const uint4* row = src + ((long long)(r.tok + x) * a.n_kv_heads + h) * (D / 8);
            vl[ps] = row[jl];
            vh[ps] = row[HV + jl];
        }
    }
    auto values = [&](int ps, float (&lo)[8], float (&hi)[8], bool first) {
        unpack<T>(vl[ps], lo);
        unpack<T>(vh[ps], hi);
        if constexpr (kK) {
            if (first) inv[ps] = a.k_norm_w ? inv_rms<D>(lo, hi, a.norm_eps) : 1.f;
            const int at = (r.tok - tok0 + min(ps * RPP + rl, r.n - 1)) * (D / 2) + 8 * jl;
            norm_rotate(lo, hi, a.k_norm_w ? wk + 8 * jl : nullptr, wk + D / 2 + 8 * jl, inv[ps],
                        a.rope ? ctab + at : nullptr, stab + at);
        }
    };
    uint32_t mx = 0u, fin = 0u;  // largest |element|, and the largest finite one, as bits
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
        if (ps * RPP >= r.n) break;  // warp-uniform
        float lo[8], hi[8];
        values(ps, lo, hi, true);
        if (ps * RPP + rl < r.n) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t x = __float_as_uint(lo[e]) & 0x7fffffffu;
                const uint32_t y = __float_as_uint(hi[e]) & 0x7fffffffu;
                mx = max(mx, max(x, y));
                if (x < 0x7f800000u) fin = max(fin, x);
                if (y < 0x7f800000u) fin = max(fin, y);
            }
        }
    }
    const bool bad = __any_sync(kFull, mx >= 0x7f800000u);  // it does not set the scale
    mx = __reduce_max_sync(kFull, fin);
    const int bpp = a.page_size / kChunk;
    const long long blk = r.blk + (long long)h * bpp;  // [page][head][block]
    uint8_t* pool = (kK ? a.k_pool : a.v_pool) + blk * (kChunk * D);
    uint8_t* scale = a.scales + blk * 2 + (kK ? 0 : 1);
    int e = kv8_need_exp(__uint_as_float(mx));
    if (r.lo > 0) {
        const int old = kv8_clamp_exp((int)*scale - 127);
        if (e > old) {
            // earlier rows of the block to the larger scale (exact above e4m3's
            // smallest normal value)
            const float f = exp2i(old - e);
            uint32_t* w = reinterpret_cast<uint32_t*>(pool);
            for (int x = lane; x < r.lo * D / 4; x += 32) {
                uint32_t h0, h1;
                e4m3x4_to_h2(w[x], h0, h1);
                const float2 p = __half22float2(*reinterpret_cast<__half2*>(&h0));
                const float2 q = __half22float2(*reinterpret_cast<__half2*>(&h1));
                w[x] = f2_to_e4m3x2(p.x * f, p.y * f) | f2_to_e4m3x2(q.x * f, q.y * f) << 16;
            }
        } else {
            e = old;
        }
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *scale = (uint8_t)(e + 127);
    const float up = exp2i(-e);
#pragma unroll
    for (int ps = 0; ps < PASSES; ++ps) {
        const int x = ps * RPP + rl;
        if (x < r.n) {
            float lo[8], hi[8];
            values(ps, lo, hi, false);
            uint2* row = reinterpret_cast<uint2*>(pool + (r.lo + x) * D);
            row[jl] = quantise8(lo, up, bad);
            row[HV + jl] = quantise8(hi, up, bad);
        }
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 3)
kv8_append_kernel(const __grid_constant__ Kv8AppendArgs a, int span, uint32_t* status,
                  uint32_t* flags) {
    constexpr int HALF = D / 2, HV = D / 16;
    __shared__ float ctab[kMaxSpan * HALF], stab[kMaxSpan * HALF];
    __shared__ float wq[D], wk[D];
    __shared__ int s_pos[kMaxSpan];
    __shared__ Run s_runs[kMaxSpan];
    __shared__ int s_first, s_end, s_nruns;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int base = blockIdx.x * span;  // the CTA's leaders: tokens base .. base + span - 1

    pdl_wait();
    if (a.q_norm_w || a.k_norm_w) {
        for (int x = tid; x < D; x += kThreads) {
            const T* q = static_cast<const T*>(a.q_norm_w);
            const T* k = static_cast<const T*>(a.k_norm_w);
            wq[x] = q ? (float)q[x] : 1.f;
            wk[x] = k ? (float)k[x] : 1.f;
        }
    }
    if (warp == 0) {
        // token base + lane and the one before it; the last one a CTA can own
        // is base + span + 14, so lane 31 sees the next CTA's first leader
        const int i = base + lane;
        const bool in = i < a.n_tokens;
        const int pos = in ? a.positions[i] : -1;
        const int seq = in ? (a.seq_ids ? a.seq_ids[i] : i) : -1;
        int ppos = __shfl_up_sync(kFull, pos, 1), pseq = __shfl_up_sync(kFull, seq, 1);
        if (lane == 0) {
            ppos = base > 0 ? a.positions[base - 1] : -1;
            pseq = base > 0 ? (a.seq_ids ? a.seq_ids[base - 1] : base - 1) : -1;
        }
        const bool cont = in && pos > 0 && ppos >= 0 && pseq == seq && pos - 1 == ppos &&
                          (pos & (kChunk - 1)) != 0;
        // tokens past the last one end the last run
        const unsigned lead = __ballot_sync(kFull, !cont);
        const int first = __ffs(lead & (span == 16 ? 0xffffu : (1u << span) - 1u)) - 1;
        const unsigned after = lead >> span << span;
        const int end = min(after ? __ffs(after) - 1 : 32, a.n_tokens - base);
        const bool mine = first >= 0 && lane >= first && lane < end;
        // runs of the CTA: leaders among its tokens that are appended
        bool use = false;
        uint32_t skipped = 0;
        Run r = {0, 0, 0, 0};
        if (mine && !cont && pos >= 0) {
            const unsigned next = lead & ~((2u << lane) - 1u);
            r.tok = i;
            r.n = min(next ? __ffs(next) - 1 : 32, end) - lane;
            r.lo = pos & (kChunk - 1);
            const int col = pos / a.page_size;
            // the positions of one block must form one run: a run that goes on
            // in the block of the token before it is refused
            const bool again = ppos >= 0 && pseq == seq && ppos / kChunk == pos / kChunk;
            uint32_t bits = 0;
            int page = 0;
            if (seq < 0 || seq >= a.n_seqs) bits = PKV_DEV_BAD_SEQ;
            else if (col >= a.table_stride || again) bits = PKV_DEV_BAD_LEN;
            else {
                page = a.table[(long long)seq * a.table_stride + col];
                if (page < 0 || page >= a.num_pages) bits = PKV_DEV_BAD_PAGE;
            }
            use = bits == 0;
            skipped = bits;
            r.blk = (long long)page * a.n_kv_heads * (a.page_size / kChunk) +
                    (pos % a.page_size) / kChunk;
        }
        skipped = __reduce_or_sync(kFull, skipped);
        if (lane == 0) {
            if (flags) flags[blockIdx.x] = skipped;
            else if (skipped) set_status(status, skipped);
        }
        const unsigned used = __ballot_sync(kFull, use);
        if (use) s_runs[__popc(used & ((1u << lane) - 1u))] = r;
        if (mine) s_pos[lane - first] = pos;
        if (lane == 0) {
            s_first = first;
            s_end = end;
            s_nruns = __popc(used);
        }
    }
    __syncthreads();
    if (s_first < 0 || s_end <= s_first) return;  // all its tokens belong to the CTA before
    const int tok0 = base + s_first;
    const int ntok = s_end - s_first;
    if (a.rope) {
        for (int x = tid; x < ntok * HALF; x += kThreads) {
            const int tk = x / HALF;
            turn_cos_sin(s_pos[tk], a.turns[x - tk * HALF], &ctab[x], &stab[x]);
        }
        __syncthreads();
    }
    // K and V blocks
    const int nruns = s_nruns;
    const int per_run = a.n_kv_heads * 2;
    for (int x = warp; x < nruns * per_run; x += kThreads / 32) {
        const int ri = x / per_run, y = x - ri * per_run;
        const Run r = s_runs[ri];
        if (y & 1) append_block<T, D, false>(a, r, y >> 1, tok0, ctab, stab, wk, lane);
        else append_block<T, D, true>(a, r, y >> 1, tok0, ctab, stab, wk, lane);
    }
    // q rows: HV lanes each
    if (a.q) {
        const uint4* q = static_cast<const uint4*>(a.q);
        uint4* qo = static_cast<uint4*>(a.q_out);
        const long long row0 = (long long)tok0 * a.n_q_heads;
        const int rows = ntok * a.n_q_heads;
        const int jl = lane % HV;
        constexpr int STEP = kThreads / HV, U = 4;  // rows a pass of the CTA; passes in flight
        for (int r0 = warp * (32 / HV) + lane / HV; r0 - lane / HV < rows; r0 += U * STEP) {
            uint4 vl[U], vh[U];
#pragma unroll
            for (int x = 0; x < U; ++x) {
                vl[x] = vh[x] = make_uint4(0u, 0u, 0u, 0u);
                const int r = r0 + x * STEP;
                if (r < rows) {
                    const uint4* row = q + (row0 + r) * (D / 8);
                    vl[x] = row[jl];
                    vh[x] = row[HV + jl];
                }
            }
#pragma unroll
            for (int x = 0; x < U; ++x) {
                const int r = r0 + x * STEP;
                if (r - lane / HV >= rows) break;  // warp-uniform
                float lo[8], hi[8];
                unpack<T>(vl[x], lo);
                unpack<T>(vh[x], hi);
                const float inv = a.q_norm_w ? inv_rms<D>(lo, hi, a.norm_eps) : 1.f;
                if (r >= rows) continue;
                const int c = r / a.n_q_heads * HALF + 8 * jl;
                norm_rotate(lo, hi, a.q_norm_w ? wq + 8 * jl : nullptr, wq + HALF + 8 * jl, inv,
                            a.rope ? ctab + c : nullptr, stab + c);
                uint4* row = qo + (row0 + r) * (D / 8);
                row[jl] = pack<T>(lo);
                row[HV + jl] = pack<T>(hi);
            }
        }
    }
    pdl_trigger();
}

}  // namespace

static int append_span(int n_tokens) { return n_tokens <= 2048 ? 1 : 16; }

int kv8_append_ctas(int n_tokens) {
    const int span = append_span(n_tokens);
    return n_tokens / span + (n_tokens % span ? 1 : 0);
}

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, int head_dim, uint32_t* status,
                              uint32_t* flags, cudaStream_t stream) {
    if (a.n_tokens <= 0) return cudaSuccess;
    const int span = append_span(a.n_tokens);
    const dim3 grid((unsigned)kv8_append_ctas(a.n_tokens));
#define PKV_KV8_APPEND(T, D) \
    return launch_pdl(kv8_append_kernel<T, D>, grid, dim3(kThreads), 0, stream, a, span, status, \
                      flags)
    if (a.bf16) {
        if (head_dim == 128) PKV_KV8_APPEND(__nv_bfloat16, 128);
        PKV_KV8_APPEND(__nv_bfloat16, 64);
    }
    if (head_dim == 128) PKV_KV8_APPEND(__half, 128);
    PKV_KV8_APPEND(__half, 64);
#undef PKV_KV8_APPEND
}

}  // namespace pkv
