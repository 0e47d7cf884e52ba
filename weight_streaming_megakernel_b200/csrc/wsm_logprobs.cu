// wsm_logprobs.cu -- log probabilities of given tokens, the entropy of their distributions and the likeliest
// alternatives (wsm_token_logprobs), what a step does with the logits of its vocabulary projection.
//
// With m = max x, y_j = (x_j - m) log2 e, l = sum 2^y_j and u = sum 2^y_j y_j, all in one pass:
//     logprob(t) = (x_t - m) - ln 2 log2 l,    entropy = ln 2 (log2 l - u / l).
// A thread keeps m, l and u of its elements and rescales them when its maximum moves; parts join exactly by
// the same rule.  The alternatives come from the same pass: each warp keeps its best 32 in order, one to a
// lane, and an element is looked at again only if it beats the warp's k-th best (and the block's best k-th).
//
// What bounds it is reading the logits once.  A row goes to one block, or with few rows to a cluster of up
// to eight, whose parts meet in the first one's shared memory: no scratch and one launch.
#include "wsm_ops.cuh"

#include <algorithm>
#include <cmath>

namespace wsm {

namespace {

static __device__ int g_logprobs_status[kOpStatusInts];

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kMaxTop = 32;         // one alternative per lane of a warp's list
constexpr int kLpUnroll = 4;        // 16-byte loads of a thread's block of elements
constexpr int kMaxCluster = 8;      // the portable cluster size

constexpr float kLog2e = 1.44269504088896341f;
constexpr float kLn2 = 0.693147180559945309f;

struct LogprobsParams {
    const void *logits;
    const long long *tokens;
    float *logprob, *entropy, *top_logprobs;
    long long *top_ids;
    long long stride;
    int rows, vocab, top;
    int ctas;                       // blocks per row
};

// Running statistics of some of a row's elements: the largest so far (-infinity: none yet), l and u relative
// to it.  Differences are taken before the factor log2 e: the type's lowest value times it is not a number.
struct Stat {
    float m, l, u;
};
// l and u move to a larger maximum; nothing summed so far (or a weight that vanishes) leaves nothing.
__device__ __forceinline__ void rebase(float &l, float &u, float from, float to) {
    const float d = fmaxf((from - to) * kLog2e, -200.f), f = ex2(d);
    u = (u + l * d) * f;
    l *= f;
}
__device__ __forceinline__ Stat join(Stat a, Stat b) {
    Stat s;
    s.m = fmaxf(a.m, b.m);
    if (a.m < s.m) rebase(a.l, a.u, a.m, s.m);
    if (b.m < s.m) rebase(b.l, b.u, b.m, s.m);
    s.l = a.l + b.l;
    s.u = a.u + b.u;
    return s;
}

// Order-preserving key of a value and its place: larger value first, then the lower index.  -0 is 0; 0 is no
// element's key.
__device__ __forceinline__ unsigned long long key_of(float x, int index) {
    const uint32_t b = __float_as_uint(x + 0.f);
    const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return ((unsigned long long)o << 32) | (0xffffffffu - (uint32_t)index);
}
__device__ __forceinline__ float key_value(unsigned long long k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return o == 0u ? -INFINITY : __uint_as_float((o & 0x80000000u) ? (o & 0x7fffffffu) : ~o);
}

// A warp's best elements, best first, one to a lane.
struct TopList {
    unsigned long long key;         // this lane's entry, 0: none
    float least;                    // value of the k-th entry (-infinity while there are fewer)
    int k;
    __device__ __forceinline__ void insert(unsigned long long cand) {
        const int pos = __popc(__ballot_sync(0xffffffffu, key > cand));
        const unsigned long long up = __shfl_up_sync(0xffffffffu, key, 1);
        const int lane = threadIdx.x & 31;
        key = lane < pos ? key : (lane == pos ? cand : up);
        least = key_value(__shfl_sync(0xffffffffu, key, k - 1));
    }
    // Offer one element per lane (want: this lane has one to offer), lanes in order.
    __device__ __forceinline__ void offer(bool want, float x, int index) {
        uint32_t todo = __ballot_sync(0xffffffffu, want);
        while (todo) {
            const int src = __ffs((int)todo) - 1;
            todo &= todo - 1;
            const float v = __shfl_sync(0xffffffffu, x, src);
            if (v < least) continue;                    // the list has moved on
            insert(key_of(v, __shfl_sync(0xffffffffu, index, src)));
        }
    }
};

// The k-th largest of the warp's 32 values.
__device__ __forceinline__ float kth_of_warp(float v, int k) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1) {
#pragma unroll
        for (int j = size >> 1; j > 0; j >>= 1) {
            const float w = __shfl_xor_sync(0xffffffffu, v, j);
            const bool desc = (lane & size) == 0, low = (lane & j) == 0;
            v = (low == desc) ? fmaxf(v, w) : fminf(v, w);
        }
    }
    return __shfl_sync(0xffffffffu, v, k - 1);
}

template <typename T, int VEC> __device__ __forceinline__ void unpack_vec(const uint4 &v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (VEC == 4) {
            x[i] = __uint_as_float(w[i]);
        } else {
            const float2 f = unpack2<T>(w[i]);
            x[2 * i] = f.x;
            x[2 * i + 1] = f.y;
        }
    }
}

template <typename T, bool kTop>
__global__ void __launch_bounds__(kLpThreads, 2) logprobs_kernel(const __grid_constant__ LogprobsParams p) {
    constexpr int VEC = 16 / (int)sizeof(T);
    constexpr int NB = kLpUnroll * VEC;                 // elements of a thread's block
    __shared__ Stat warp_stat[kLpWarps];
    __shared__ unsigned long long warp_top[kTop ? kLpWarps : 1][kMaxTop];
    __shared__ unsigned long long best[kMaxTop];
    // what the row's blocks bring to the first one
    __shared__ Stat all_stat[kMaxCluster];
    __shared__ unsigned long long all_top[kTop ? kMaxCluster : 1][kMaxTop];
    __shared__ int shared_least;                        // order-preserving bits of the warps' best k-th value

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = p.ctas > 1 ? (int)cluster_ctarank() : 0;
    const long long row = (long long)blockIdx.x / p.ctas;
    if (kTop && threadIdx.x < kMaxTop) best[threadIdx.x] = 0ull;
    if (threadIdx.x == 0) shared_least = (int)0x80000000;
    __syncthreads();
    if (p.ctas > 1) cluster_sync_all();                 // every block of the row is there to be written to
    pdl_wait();
    pdl_launch_dependents();

    // The row: elements before the first 16-byte boundary, whole vectors (dealt to the row's blocks in
    // consecutive stretches), and the rest.
    const T *x_row = reinterpret_cast<const T *>(p.logits) + row * p.stride;
    const int head = min(p.vocab, (int)(((16u - (uint32_t)(reinterpret_cast<uintptr_t>(x_row) & 15u)) & 15u) / sizeof(T)));
    const int n_vec = (p.vocab - head) / VEC;
    const int tail0 = head + n_vec * VEC;
    const int share = (n_vec + p.ctas - 1) / p.ctas;
    const int v_begin = min(n_vec, part * share), v_end = min(n_vec, v_begin + share);
    const uint4 *vec = reinterpret_cast<const uint4 *>(x_row + head);

    Stat st = {-INFINITY, 0.f, 0.f};
    float base = 0.f;                                   // what y is counted from: the largest so far, or 0
    TopList top;
    top.key = 0ull;
    top.least = -INFINITY;
    top.k = p.top;

    auto raise = [&](float bm) {                        // bm > st.m: the maximum moves
        rebase(st.l, st.u, st.m, bm);
        st.m = base = bm;
    };
    auto add = [&](float x, float &l, float &u) {
        const float y = (x - base) * kLog2e;
        const float e = ex2(y);
        l += e;
        u = fmaf(e, fmaxf(y, -200.f), u);               // (-infinity: weight 0 times a finite number)
    };
    auto single = [&](bool have, int index) {           // one element per lane: a row's ragged ends
        const float x = have ? to_f32<T>(x_row[index]) : -INFINITY;
        if (x > st.m) raise(x);
        add(x, st.l, st.u);
        if constexpr (kTop) top.offer(x > top.least, x, index);
    };
    if (part == 0 && warp == 0 && head > 0) single(lane < head, lane);

    uint4 cur[kLpUnroll];
    constexpr int kStep = kLpThreads * kLpUnroll;       // vectors a block takes per turn
    // a warp's vectors ascend from turn to turn and, within one, from load to load
    int v0 = v_begin + warp * (32 * kLpUnroll) + lane;
    auto load = [&](int at, uint4 (&r)[kLpUnroll]) {
#pragma unroll
        for (int i = 0; i < kLpUnroll; ++i)
            if (at + i * 32 < v_end) r[i] = __ldcs(vec + at + i * 32);
    };
    load(v0, cur);
    bool fresh = true;                                  // no block of this warp seen yet
    const int turns = (v_end - v_begin + kStep - 1) / kStep;
    for (int turn = 0; turn < turns; ++turn) {
        uint4 next[kLpUnroll];
        load(v0 + kStep, next);
        float x[NB];
#pragma unroll
        for (int i = 0; i < kLpUnroll; ++i) {
            if (v0 + i * 32 < v_end) {
                unpack_vec<T, VEC>(cur[i], &x[i * VEC]);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) x[i * VEC + j] = -INFINITY;
            }
        }
        float bm = x[0];
#pragma unroll
        for (int j = 1; j < NB; ++j) bm = fmaxf(bm, x[j]);
        if (bm > st.m) raise(bm);
        float l = 0.f, u = 0.f;                         // the block's own sums first: shorter chains of roundings
#pragma unroll
        for (int j = 0; j < NB; ++j) add(x[j], l, u);
        st.l += l;
        st.u += u;
        if constexpr (kTop) {
            // Candidates beat the warp's k-th value as it was before this turn: an equal one comes later in
            // the row than all that are listed.  Against another warp's k-th an equal one may still win.
            float over = top.least;
            float from = over;
            const int sl = *(volatile int *)&shared_least;
            if (sl != (int)0x80000000) from = fmaxf(from, __int_as_float(sl < 0 ? sl ^ 0x7fffffff : sl));
            if (fresh) {
                // the k-th largest of the lanes' maxima is a floor for the k-th element
                from = fmaxf(from, kth_of_warp(bm, p.top));
                fresh = false;
            }
            if (__any_sync(0xffffffffu, bm > over && bm >= from)) {
#pragma unroll
                for (int j = 0; j < NB; ++j)
                    top.offer(x[j] > over && x[j] >= from, x[j],
                              head + (v0 + (j / VEC) * 32) * VEC + (j % VEC));
                if (lane == 0 && top.least > -INFINITY) {
                    const int b = __float_as_int(top.least + 0.f);
                    atomicMax(&shared_least, b < 0 ? b ^ 0x7fffffff : b);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < kLpUnroll; ++i) cur[i] = next[i];
        v0 += kStep;
    }
    if (part == p.ctas - 1 && warp == kLpWarps - 1 && tail0 < p.vocab)
        single(tail0 + lane < p.vocab, tail0 + lane);

    // ---- the warp's, the block's, the row's statistics
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        Stat b;
        b.m = __shfl_xor_sync(0xffffffffu, st.m, o);
        b.l = __shfl_xor_sync(0xffffffffu, st.l, o);
        b.u = __shfl_xor_sync(0xffffffffu, st.u, o);
        st = join(st, b);
    }
    if (lane == 0) warp_stat[warp] = st;
    if constexpr (kTop) warp_top[warp][lane] = lane < p.top ? top.key : 0ull;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kLpWarps; ++w) st = join(st, warp_stat[w]);
        if (part == 0) {
            all_stat[0] = st;
        } else {
            const uint32_t a = map_to_rank(smem_u32(&all_stat[part]), 0);
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(st.m) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 4), "f"(st.l) : "memory");
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a + 8), "f"(st.u) : "memory");
        }
    }
    if constexpr (kTop) {
        // an entry's place is the number of larger ones (no two are equal); the best p.top of the block
        const unsigned long long mine = warp_top[warp][lane];
        int rank = 0;
        for (int w = 0; w < kLpWarps; ++w)
            for (int j = 0; j < p.top; ++j) rank += warp_top[w][j] > mine ? 1 : 0;
        if (mine != 0ull && rank < p.top) best[rank] = mine;
        __syncthreads();
        if (p.ctas > 1) {
            if (threadIdx.x < kMaxTop) {
                const uint32_t a = map_to_rank(smem_u32(&all_top[part][threadIdx.x]), 0);
                asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(best[threadIdx.x]) : "memory");
            }
        }
    }
    if (p.ctas > 1) {
        cluster_sync_all();                             // the parts are in the first block's shared memory
        if (part != 0) return;
        if constexpr (kTop) {
            const unsigned long long mine = warp < p.ctas ? all_top[warp][lane] : 0ull;
            if (threadIdx.x < kMaxTop) best[threadIdx.x] = 0ull;
            __syncthreads();
            int rank = 0;
            for (int w = 0; w < p.ctas; ++w)
                for (int j = 0; j < p.top; ++j) rank += all_top[w][j] > mine ? 1 : 0;
            if (mine != 0ull && rank < p.top) best[rank] = mine;
            __syncthreads();
        }
    }
    static_assert(kMaxCluster <= kLpWarps, "one warp per block's list");
    if (warp != 0) return;
    __syncwarp();                                       // (all_stat[0] is lane 0's own write)
    Stat s = {-INFINITY, 0.f, 0.f};
    if (lane == 0) {
        s = all_stat[0];
        for (int c = 1; c < p.ctas; ++c) s = join(s, all_stat[c]);
    }
    s.m = __shfl_sync(0xffffffffu, s.m, 0);
    s.l = __shfl_sync(0xffffffffu, s.l, 0);
    s.u = __shfl_sync(0xffffffffu, s.u, 0);
    const bool none = s.l == 0.f;                       // no element above -infinity
    const float from = none ? 0.f : s.m;
    const float log_l = none ? 0.f : log2f(s.l);
    auto logprob_of = [&](float x) { return (x - from) - log_l * kLn2; };
    if (lane == 0) {
        if (p.logprob) {
            const long long t = p.tokens ? p.tokens[row] : -1;
            float lp = 0.f;
            if (t >= p.vocab) {
                lp = NAN;
                record_op_error(g_logprobs_status, kCodeInvalid, (int)row, kSiteToken);
            } else if (t >= 0) {
                lp = logprob_of(to_f32<T>(x_row[t]));
            }
            p.logprob[row] = lp;
        }
        if (p.entropy) {
            const float h = none ? 0.f : (log_l - s.u / s.l) * kLn2;
            p.entropy[row] = h < 0.f ? 0.f : h;         // (a certain token: rounding may leave -1e-8; NaN stays)
        }
    }
    if constexpr (kTop) {
        if (lane < p.top) {
            const unsigned long long k = best[lane];
            const bool bad = s.l != s.l;
            p.top_ids[row * p.top + lane] = (k == 0ull || bad) ? -1 : (long long)(0xffffffffu - (uint32_t)k);
            p.top_logprobs[row * p.top + lane] = bad ? NAN : (k == 0ull ? -INFINITY : logprob_of(key_value(k)));
        }
    }
}

template <typename T>
wsm_status run_logprobs(const LogprobsParams &p, cudaStream_t stream) {
    const dim3 grid((unsigned)((long long)p.rows * p.ctas));
    return p.top > 0 ? op_launch(&logprobs_kernel<T, true>, grid, kLpThreads, 0, stream, p, p.ctas)
                     : op_launch(&logprobs_kernel<T, false>, grid, kLpThreads, 0, stream, p, p.ctas);
}

}  // namespace

wsm_status logprobs_status_ptr(void **p) {
    WSM_OP_CUDA(cudaGetSymbolAddress(p, g_logprobs_status));
    return WSM_OK;
}

}  // namespace wsm

using namespace wsm;

extern "C" wsm_status wsm_token_logprobs(const wsm_logprobs *a, wsm_stream_t stream_) {
    if (!a) return op_fail(WSM_ERR_INVALID, "the arguments must be non-null");
    if (a->rows < 0 || a->vocab < 1) return op_fail(WSM_ERR_INVALID, "rows %d, vocab %d: no negative sizes, and a token at least", a->rows, a->vocab);
    if (a->top < 0 || a->top > kMaxTop || a->top > a->vocab)
        return op_fail(WSM_ERR_UNSUPPORTED, "top %d: 0 to %d alternatives, no more than the vocabulary of %d", a->top, kMaxTop, a->vocab);
    if (a->vocab > (1 << 30)) return op_fail(WSM_ERR_UNSUPPORTED, "a vocabulary of %d is too large", a->vocab);
    if (a->dtype != WSM_DTYPE_FP32 && a->dtype != WSM_DTYPE_BF16 && a->dtype != WSM_DTYPE_FP16)
        return op_fail(WSM_ERR_UNSUPPORTED, "logits element type %d: fp32, bf16 and fp16 are", a->dtype);
    if (a->stride < 0) return op_fail(WSM_ERR_INVALID, "the row stride must not be negative");
    if (a->rows == 0) return WSM_OK;
    if (!a->logits) return op_fail(WSM_ERR_INVALID, "logits must be a non-null device pointer");
    if (a->top > 0 && (!a->top_ids || !a->top_logprobs))
        return op_fail(WSM_ERR_INVALID, "top_ids and top_logprobs must be non-null device pointers when top > 0");
    if (!a->logprob && !a->entropy && a->top == 0) return op_fail(WSM_ERR_INVALID, "no output was asked for");
    const size_t es = a->dtype == WSM_DTYPE_FP32 ? 4 : 2;
    if (!aligned_to(a->logits, es) || !aligned_to(a->tokens, 8) || !aligned_to(a->top_ids, 8) || !aligned_to(a->logprob, 4) ||
        !aligned_to(a->entropy, 4) || !aligned_to(a->top_logprobs, 4))
        return op_fail(WSM_ERR_ALIGN, "every pointer must be aligned to its elements");
    int dev, sms;
    wsm_status st = device_sms(&dev, &sms);
    if (st != WSM_OK) return st;
    LogprobsParams p = {};
    p.logits = a->logits;
    p.tokens = a->tokens;
    p.logprob = a->logprob;
    p.entropy = a->entropy;
    p.top_ids = a->top_ids;
    p.top_logprobs = a->top_logprobs;
    p.stride = a->stride;
    p.rows = a->rows;
    p.vocab = a->vocab;
    p.top = a->top;
    // blocks per row: as many as keep two on every SM busy, while each has a few kilobytes to read
    p.ctas = 1;
    while (p.ctas < kMaxCluster && (long long)p.rows * p.ctas * 2 <= 2ll * sms && (size_t)p.vocab * es / (2 * p.ctas) >= 4096)
        p.ctas *= 2;
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (a->dtype == WSM_DTYPE_FP32) return run_logprobs<float>(p, stream);
    return a->dtype == WSM_DTYPE_BF16 ? run_logprobs<__nv_bfloat16>(p, stream) : run_logprobs<__half>(p, stream);
}
