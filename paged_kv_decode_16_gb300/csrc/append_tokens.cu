// append_tokens.cu -- rotary embedding of new tokens' q and k (in halves or interleaved
// pairs, on part of a head, any frequencies), and the write of k and v into their slots.
//
// One pass over the rows: a task is two 16-byte vectors of one row that turn together
// (half layout: vector j and vector j + rotary_dim / 16, elements i and i + rotary_dim
// / 2; interleaved: two neighbouring vectors), so that no lane needs another's elements,
// and in both layouts the task's eight cosines and sines are those of pairs 8 j .. 8 j +
// 7.  The D / 16 tasks of a row lie on neighbouring lanes, which is where the optional
// norm sums its squares.
//
// A CTA takes groups of up to four tokens.  What a group's tasks share is worked out once,
// in shared memory, while the group in front of it runs: cosines and sines, and the
// addresses of every row (a source, and a destination with the row's kind and token in its
// low bits).  The rows come by asynchronous copies, a few tasks ahead, into places of the
// thread's own (no barrier).
//
// What bounds it: memory, 2 bytes read and 2 written an element.  14,433 tokens of 32 + 8 + 8
// rows of 128 with norms: 59.5 us, 6.0 TB/s (a copy of the same bytes: 58); without the shared
// addresses, 390 instructions a task and warp instead of 260, it was 71.  Two tasks ahead and
// four CTAs an SM: 58 to 68 us with three, 60 to 82 with four and six tasks.
#include "packed.cuh"
#include "selected.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;    // a grid is one wave of them
constexpr int kAhead = 2;        // a thread's tasks on their way
constexpr int kMaxTokens = 4;    // tokens of a group (two bits of a destination)
constexpr int kMaxRows = 1024;   // rows of a group, unless one token has more

enum Kind { kV = 0, kQ = 1, kK = 2 };  // of a row, the low bits of its destination

__device__ __forceinline__ void copy16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// (x, y) turned by the angle of (c, s).
__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
    const float a = x * c - y * s;
    y = y * c + x * s;
    x = a;
}

struct GroupShape {
    int tokens;        // of a group
    int rows;          // of a token: q, k, v
    uint32_t by_rows;  // 2^32 / rows, rounded up: r / rows for the r of a group
    int items;         // steps of kThreads tasks
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
append_tokens_kernel(const AppendTokensArgs a, const GroupShape gs) {
    constexpr int kTasks = D / 16;            // of a row
    constexpr int kRows = kThreads / kTasks;  // rows of an item
    __shared__ __align__(16) float s_cos[2][kMaxTokens][64];
    __shared__ __align__(16) float s_sin[2][kMaxTokens][64];
    __shared__ __align__(16) float s_w[2][2][D / 2];  // q's and k's norm weights, by vector
    __shared__ long long s_base[2][kMaxTokens];       // a token's row of head 0 in the pools, or -1
    __shared__ int s_pos[2][kMaxTokens];
    extern __shared__ __align__(16) uint8_t s_dyn[];
    uint4* s_ring = reinterpret_cast<uint4*>(s_dyn);  // [kAhead][2][kThreads]
    const int pad = gs.items * kRows;
    uint64_t* s_src = reinterpret_cast<uint64_t*>(s_ring + kAhead * 2 * kThreads);  // [3][pad]
    uint64_t* s_dst = s_src + 3 * pad;                                              // [2][pad]

    const int tid = threadIdx.x;
    const int groups = 1 + (a.n_tokens - 1) / gs.tokens;
    const bool rope = a.positions != nullptr;
    const bool normed = a.q_norm || a.k_norm;
    const int pairs = rope ? a.rope.rotary_dim >> 1 : 0;
    const int turning = rope ? a.rope.rotary_dim >> 4 : 0;  // tasks of a row that turn
    const int j = tid % kTasks, row0 = tid / kTasks;        // the thread's place in an item
    const bool near = a.rope.interleaved || j >= turning;   // its two vectors are neighbours
    const int v0 = (near ? 2 * j : j) * 8, v1 = (near ? 2 * j + 1 : j + turning) * 8;
    // tasks on their way: at most one group's, whose addresses are there
    const bool deep = gs.items >= kAhead;
    const int depth = deep ? kAhead : gs.items;

    auto row_of = [&](int i, int& tk) {
        tk = (int)__umulhi((uint32_t)i, gs.by_rows);
        return i - tk * gs.rows;
    };
    auto fill_src = [&](int g, int buf) {
        for (int i = tid; i < pad; i += kThreads) {
            int tk;
            const int r = row_of(i, tk);
            const long long t = (long long)g * gs.tokens + tk;
            const T* p = nullptr;
            if (tk < gs.tokens && t < a.n_tokens) {
                if (r < a.n_q_heads)
                    p = static_cast<const T*>(a.q) + t * a.q_stride + r * D;
                else if (r < a.n_q_heads + a.n_kv_heads)
                    p = static_cast<const T*>(a.k) + t * a.k_stride + (r - a.n_q_heads) * D;
                else
                    p = static_cast<const T*>(a.v) + t * a.v_stride +
                        (r - a.n_q_heads - a.n_kv_heads) * D;
            }
            s_src[buf * pad + i] = reinterpret_cast<uint64_t>(p);
        }
    };
    // What a token's rows go by: its position and its row in the pools.
    long long tok_slot = -1;
    int tok_pos = -1;
    auto read_token = [&](int g) {
        const long long t = (long long)g * gs.tokens + tid;
        tok_slot = -1;
        tok_pos = -1;
        if (tid < gs.tokens && g < groups && t < a.n_tokens) {
            tok_slot = a.slots[t];
            tok_pos = rope ? a.positions[t] : 0;
        }
    };
    auto keep_token = [&](int buf) {
        if (tid >= gs.tokens) return;
        if (tok_slot >= a.n_slots) {
            set_status(a.status, PKV_DEV_BAD_PAGE);
            tok_slot = -1;
        }
        const long long page = tok_slot / a.page_size;
        s_base[buf][tid] = tok_slot < 0 || tok_pos < 0
                               ? -1
                               : (page * a.n_kv_heads * a.page_size +
                                  (tok_slot - page * a.page_size)) * D;
        s_pos[buf][tid] = tok_pos;
    };
    // Group g's destinations, cosines and sines.
    auto fill = [&](int g, int buf) {
        for (int i = tid; i < pad; i += kThreads) {
            int tk;
            const int r = row_of(i, tk);
            uint64_t d = 0;
            if (tk < gs.tokens) {
                const long long t = (long long)g * gs.tokens + tk, base = s_base[buf][tk];
                if (r < a.n_q_heads) {
                    if (s_pos[buf][tk] >= 0)
                        d = reinterpret_cast<uint64_t>(static_cast<T*>(a.q_out) +
                                                       t * a.q_out_stride + r * D);
                    d |= kQ;
                } else {
                    const bool k = r < a.n_q_heads + a.n_kv_heads;
                    const int head = r - a.n_q_heads - (k ? 0 : a.n_kv_heads);
                    if (base >= 0)
                        d = reinterpret_cast<uint64_t>(
                            static_cast<T*>(k ? a.k_pool : a.v_pool) + base +
                            (long long)head * (a.page_size * D));
                    d |= k ? kK : kV;
                }
                d |= (uint64_t)tk << 2;
            }
            s_dst[buf * pad + i] = d;
        }
        if (tid < gs.tokens * pairs) {
            const int tk = tid / pairs, p = tid - tk * pairs, pos = s_pos[buf][tk];
            // the turns' product wraps modulo one turn by itself; its top 32 bits are a signed
            // fraction of half a turn, which fp32 then rounds (2^-26 turns at most)
            const uint64_t ph = (uint64_t)(int64_t)pos * a.rope.turns[p];
            float s, c;
            sincospif((float)(int)(ph >> 32) * 4.6566128730773926e-10f, &s, &c);
            s_cos[buf][tk][place<64>(p)] = c * a.rope.magnitude;
            s_sin[buf][tk][place<64>(p)] = s * a.rope.magnitude;
        }
    };

    int load_item = 0, load_buf = 0, stage_in = 0;
    auto load = [&]() {  // the next task's two vectors, on their way to the thread's place
        const T* src = reinterpret_cast<const T*>(s_src[load_buf * pad + load_item * kRows + row0]);
        if (src) {
            uint4* dst = s_ring + stage_in * 2 * kThreads + tid;
            copy16(dst, src + v0);
            copy16(dst + kThreads, src + v1);
        }
        copies_commit();
        if (++load_item == gs.items) {
            load_item = 0;
            load_buf = load_buf == 2 ? 0 : load_buf + 1;
        }
        if (++stage_in == depth) stage_in = 0;
    };

    fill_src(blockIdx.x, 0);
    fill_src(blockIdx.x + gridDim.x, 1);
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    read_token(blockIdx.x);
    for (int u = 0; u < depth; ++u) load();
    if (normed && tid < 2 * kTasks) {
        const T* w = static_cast<const T*>(tid < kTasks ? a.q_norm : a.k_norm);
        float f[8], h[8];
        if (w) {
            Cvt<T>::unpack8(*reinterpret_cast<const uint4*>(w + v0), f);
            Cvt<T>::unpack8(*reinterpret_cast<const uint4*>(w + v1), h);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                s_w[tid / kTasks][0][place<D / 2>(8 * j + e)] = f[e];
                s_w[tid / kTasks][1][place<D / 2>(8 * j + e)] = h[e];
            }
        }
    }
    keep_token(0);
    __syncthreads();
    fill(blockIdx.x, 0);
    read_token(blockIdx.x + gridDim.x);
    keep_token(1);

    int stage = 0, buf = 0, src_buf = 2;
    for (int g = blockIdx.x; g < groups; g += gridDim.x, buf ^= 1) {
        __syncthreads();  // what this group goes by is there; the last group's readers are done
        const bool more = g + gridDim.x < groups;
        if (more) {
            fill_src(g + 2 * gridDim.x, src_buf);
            src_buf = src_buf == 2 ? 0 : src_buf + 1;
            fill(g + gridDim.x, buf ^ 1);
            read_token(g + 2 * gridDim.x);
        }
        for (int item = 0; item < gs.items; ++item) {
            if (deep) copies_wait<kAhead - 1>();
            else copies_wait<0>();
            const uint64_t d = s_dst[buf * pad + item * kRows + row0];
            const int kind = (int)d & 3, tk = (int)(d >> 2) & 3;
            uint4* ring = s_ring + stage * 2 * kThreads + tid;
            uint4 x = ring[0], y = ring[kThreads];
            const bool turn = kind != kV && j < turning;
            const bool norm = kind == kQ ? a.q_norm != nullptr : kind == kK && a.k_norm != nullptr;
            if (__any_sync(kFull, turn || norm)) {
                f2 f[4], h[4];
                unpack<T>(x, f);
                unpack<T>(y, h);
                if (normed) {
                    f2 sum2 = mul2(f[0], f[0]);
#pragma unroll
                    for (int e = 1; e < 4; ++e) sum2 = fma2(f[e], f[e], sum2);
#pragma unroll
                    for (int e = 0; e < 4; ++e) sum2 = fma2(h[e], h[e], sum2);
                    float sum, other;
                    split_f2(sum2, sum, other);
                    sum += other;
#pragma unroll
                    for (int o = kTasks / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
                    if (norm) {
                        const float inv = rsqrtf(fmaf(sum, 1.0f / (float)D, a.eps));
                        const f2 inv2 = make_f2(inv, inv);
                        f2 w[4];
                        load8<D / 2>(s_w[kind - 1][0], j, w);
#pragma unroll
                        for (int e = 0; e < 4; ++e) f[e] = mul2(mul2(f[e], inv2), w[e]);
                        load8<D / 2>(s_w[kind - 1][1], j, w);
#pragma unroll
                        for (int e = 0; e < 4; ++e) h[e] = mul2(mul2(h[e], inv2), w[e]);
                    }
                }
                if (turn) {
                    f2 c[4], s[4];
                    load8<64>(s_cos[buf][tk], j, c);
                    load8<64>(s_sin[buf][tk], j, s);
                    if (a.rope.interleaved) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            // elements 2 i and 2 i + 1 are one pair of floats
                            f2(&z)[4] = e < 2 ? f : h;
                            float c0, c1, s0, s1, p0, p1, q0, q1;
                            split_f2(c[e], c0, c1);
                            split_f2(s[e], s0, s1);
                            split_f2(z[e % 2 * 2], p0, p1);
                            split_f2(z[e % 2 * 2 + 1], q0, q1);
                            turn_pair(p0, p1, c0, s0);
                            turn_pair(q0, q1, c1, s1);
                            z[e % 2 * 2] = make_f2(p0, p1);
                            z[e % 2 * 2 + 1] = make_f2(q0, q1);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const f2 z = fma2(f[e], c[e], neg2(mul2(h[e], s[e])));
                            h[e] = fma2(f[e], s[e], mul2(h[e], c[e]));
                            f[e] = z;
                        }
                    }
                }
                if (turn || norm) {
                    x = pack<T>(f);
                    y = pack<T>(h);
                }
            }
            T* dst = reinterpret_cast<T*>(d & ~15ull);
            if (dst) {
                *reinterpret_cast<uint4*>(dst + v0) = x;
                *reinterpret_cast<uint4*>(dst + v1) = y;
            }
            load();  // into the place just read (behind the last group: nothing)
            if (++stage == depth) stage = 0;
        }
        if (more) keep_token(buf);
    }
    copies_wait<0>();
}

template <typename T, int D>
cudaError_t launch(const AppendTokensArgs& a, cudaStream_t stream) {
    constexpr int kItemRows = kThreads / (D / 16);
    const int ctas = kCtasPerSm * sm_count();
    // a token a CTA while that is one wave, then groups of up to kMaxTokens
    GroupShape gs;
    gs.rows = a.n_q_heads + 2 * a.n_kv_heads;
    gs.tokens = 1 + (a.n_tokens - 1) / ctas;
    if (gs.tokens > kMaxTokens) gs.tokens = kMaxTokens;
    while (gs.tokens > 1 && gs.tokens * gs.rows > kMaxRows) --gs.tokens;
    gs.by_rows = (uint32_t)(((1ull << 32) + gs.rows - 1) / gs.rows);
    gs.items = (gs.tokens * gs.rows + kItemRows - 1) / kItemRows;
    const int groups = 1 + (a.n_tokens - 1) / gs.tokens;
    constexpr int kRing = kAhead * 2 * kThreads * 16;
    static SmemLimit limit;
    const cudaError_t e = limit.set(reinterpret_cast<const void*>(append_tokens_kernel<T, D>),
                                    kRing + 5 * 8 * (kMaxAppendRows + kItemRows));
    if (e != cudaSuccess) return e;
    return launch_pdl(append_tokens_kernel<T, D>, dim3(groups < ctas ? groups : ctas),
                      dim3(kThreads), kRing + 5 * 8 * gs.items * kItemRows, stream, a, gs);
}

}  // namespace

cudaError_t launch_append_tokens(const AppendTokensArgs& a, bool bf16, int head_dim,
                                 cudaStream_t stream) {
    if (bf16)
        return head_dim == 128 ? launch<__nv_bfloat16, 128>(a, stream)
                               : launch<__nv_bfloat16, 64>(a, stream);
    return head_dim == 128 ? launch<__half, 128>(a, stream) : launch<__half, 64>(a, stream);
}

}  // namespace pkv
