// wsm_logprobs.cu -- log probabilities of given tokens, the entropy of their distributions and the likeliest
// alternatives (wsm_token_logprobs), what a step does with the logits of its vocabulary projection.
//
// With m = max x, y_j = (x_j - m) log2 e, l = sum 2^y_j and u = sum 2^y_j y_j, all in one pass:
//     logprob(t) = (x_t - m) - ln 2 log2 l,    entropy = ln 2 (log2 l - u / l).
// A thread keeps m, l and u of its elements and rescales them when its maximum moves; parts join exactly by
// the same rule.
//
// The alternatives: at least k elements reach the k-th largest of the block's 256 threads' maxima, and few more
// do.  A thread remembers where its maximum was and how large its other blocks got, so after the pass the threads
// that reach that floor read one block of theirs again (now and then all of them), and the elements found are
// ranked by counting.  Where that finds too many -- thousands of equal values, or nearly all of a row masked --
// the block goes through its part once more with a sorted list of the best 32 in each warp's lanes, which is
// slower and has no such case.
//
// What bounds it is reading the logits once.  A row goes to one block, or with few rows to a cluster of up
// to eight, whose parts meet in the first one's shared memory: no scratch and one launch.
//
// Measured on a B200: 2049 rows of 100003 fp32 126 to 136 us, 6.0 to 6.5 TB/s (a copy moves 6.44); 128 rows of
// 128000 bf16, 20 alternatives, 17 us (floor 5.1) and 4 rows of 131072 fp32, 8 alternatives, 8.5 to 9 us (0.3): a read's
// latency, the pass, then some 3 us to find and rank the alternatives.
#include "wsm_ops.cuh"

#include <algorithm>
#include <cmath>

namespace wsm {

namespace {

static __device__ unsigned long long g_logprobs_error;

constexpr int kLpThreads = 256;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kMaxTop = 32;         // one alternative per lane of a warp's list
// 16-byte loads of a thread in a turn over the row.  Where every SM has a block or two, many loads to each; with more
// rows fewer, for three blocks to an SM: what follows a row's pass (its alternatives, some 3 us) hides behind the
// others' passes.  (On a B200, 8 loads and two blocks, 4 and three: 128 rows of 128000 bf16, nine in ten masked, 17
// and 20 us, 148 rows of 128000 fp32 without alternatives 14 and 16; 391 rows of 102912 fp32 with 32 alternatives 50
// and 39, 707 of 3405 with 5 18 and 13, 412 of 34409 fp16 22 and 14.)
constexpr int kFewRowsLoads = 8, kManyRowsLoads = 4;
constexpr int kLpUnroll = 4;        // ... and how many of them it unpacks at a time
constexpr int kFound = 512;         // elements that reach the floor there is room for
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

// Running statistics of some of a row's elements: the largest so far (-infinity: none yet), and l and u relative
// to r = m log2 e, rounded: y is one operation, x log2 e - r, off by the same rounding for all elements, which
// logprobs take back.  For a maximum past kFar that rounding would no longer be small (nor r a number, for the
// type's lowest value); there elements go by far_y, two operations.
constexpr float kFar = 65536.f;
struct Stat {
    float m, r, l, u;
};
// (rounded by itself: contracted with a sum it would be another number in every place)
__device__ __forceinline__ float base_of(float m) { return __fmul_rn(fminf(fmaxf(m, -kFar), kFar), kLog2e); }
// y of an element by a maximum past kFar: differences of the elements themselves, as anything else vanishes
__device__ __forceinline__ float far_y(float x, float m) { return (x - m) * kLog2e; }
// What the rounding of r adds to every y by a maximum of m: up to 2^-8 next to kFar, nothing past it.
__device__ __forceinline__ float y_offset(float m) { return fabsf(m) > kFar ? 0.f : fmaf(m, kLog2e, -base_of(m)); }
// l and u move to a larger maximum; nothing summed so far (or a weight that vanishes) leaves nothing.
__device__ __forceinline__ void rebase(Stat &s, float m) {
    const float r = base_of(m);
    float d = s.r - r;
    // (across the border: what one side's rounding added is taken off, what the other's adds put on; with nothing summed
    // so far any d will do)
    if (fabsf(m) > kFar || (fabsf(s.m) > kFar && s.m > -INFINITY)) d = far_y(s.m, m) + (y_offset(m) - y_offset(s.m));
    d = fmaxf(d, -200.f);
    const float f = ex2(d);
    s.u = (s.u + s.l * d) * f;
    s.l *= f;
    s.m = m;
    s.r = r;
}
__device__ __forceinline__ Stat no_elements() { return Stat{-INFINITY, -kFar * kLog2e, 0.f, 0.f}; }

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

// The largest of a vector's elements (NaN left aside), and a vector of -infinities.
template <typename T> struct Vec16;
template <> struct Vec16<float> {
    static constexpr uint32_t kNone = 0xff800000u;
    static __device__ __forceinline__ float max_of(const uint4 (&v)[kLpUnroll]) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < kLpUnroll; ++i)
            m = fmaxf(m, fmaxf(fmaxf(__uint_as_float(v[i].x), __uint_as_float(v[i].y)),
                               fmaxf(__uint_as_float(v[i].z), __uint_as_float(v[i].w))));
        return m;
    }
};
template <typename T2> __device__ __forceinline__ T2 word_as(uint32_t w) { return *reinterpret_cast<T2 *>(&w); }
template <typename T2> __device__ __forceinline__ T2 max_of_words(const uint4 (&v)[kLpUnroll]) {
    T2 m = word_as<T2>(v[0].x);
#pragma unroll
    for (int i = 0; i < kLpUnroll; ++i)
        m = __hmax2(m, __hmax2(__hmax2(word_as<T2>(v[i].x), word_as<T2>(v[i].y)), __hmax2(word_as<T2>(v[i].z), word_as<T2>(v[i].w))));
    return m;
}
template <> struct Vec16<__nv_bfloat16> {
    static constexpr uint32_t kNone = 0xff80ff80u;
    static __device__ __forceinline__ float max_of(const uint4 (&v)[kLpUnroll]) {
        const float2 f = __bfloat1622float2(max_of_words<__nv_bfloat162>(v));
        return fmaxf(f.x, f.y);
    }
};
template <> struct Vec16<__half> {
    static constexpr uint32_t kNone = 0xfc00fc00u;
    static __device__ __forceinline__ float max_of(const uint4 (&v)[kLpUnroll]) {
        const float2 f = __half22float2(max_of_words<__half2>(v));
        return fmaxf(f.x, f.y);
    }
};

// Where a block's part of a row lies: elements before the first 16-byte boundary (the first block's), whole
// vectors (dealt to the row's blocks in consecutive stretches), and the rest (the last block's).
template <typename T, int kLpLoads> struct RowPart {
    static constexpr int VEC = 16 / (int)sizeof(T);
    static constexpr int kStep = kLpThreads * kLpLoads; // vectors a block takes per turn
    const T *x;
    const uint4 *vec;
    int head, tail0, vocab, v_begin, v_end, turns;
    bool first, last;
    __device__ __forceinline__ RowPart(const LogprobsParams &p, long long row, int part) {
        x = reinterpret_cast<const T *>(p.logits) + row * p.stride;
        vocab = p.vocab;
        head = min(vocab, (int)(((16u - (uint32_t)(reinterpret_cast<uintptr_t>(x) & 15u)) & 15u) / sizeof(T)));
        const int n_vec = (vocab - head) / VEC;
        tail0 = head + n_vec * VEC;
        const int share = (n_vec + p.ctas - 1) / p.ctas;
        v_begin = min(n_vec, part * share);
        v_end = min(n_vec, v_begin + share);
        vec = reinterpret_cast<const uint4 *>(x + head);
        turns = (v_end - v_begin + kStep - 1) / kStep;
        first = part == 0;
        last = part == p.ctas - 1;
    }
    // load i of a thread in a turn: a warp's vectors ascend from turn to turn and from load to load
    __device__ __forceinline__ int vector_at(int turn, int i) const {
        return v_begin + turn * kStep + (int)(threadIdx.x >> 5) * (32 * kLpLoads) + i * 32 + (int)(threadIdx.x & 31);
    }
};

// Whole numbers in the order of the values (-0 is 0), and back.
__device__ __forceinline__ int ordered_int(float x) {
    const int b = __float_as_int(x + 0.f);
    return b < 0 ? b ^ 0x7fffffff : b;
}
__device__ __forceinline__ float from_ordered(int b) { return __int_as_float(b < 0 ? b ^ 0x7fffffff : b); }

// The best p.top of a block's part by sorted lists: every element is offered to its warp's.  Leaves them in
// best[], best first.  All threads.
template <typename T, int kLpLoads>
__device__ __noinline__ void top_by_lists(const RowPart<T, kLpLoads> &r, int k, unsigned long long (*warp_top)[kMaxTop],
                                          unsigned long long *best) {
    constexpr int VEC = RowPart<T, kLpLoads>::VEC;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    TopList top;
    top.key = 0ull;
    top.least = -INFINITY;
    top.k = k;
    auto single = [&](bool have, int index) {
        const float x = have ? to_f32<T>(r.x[index]) : -INFINITY;
        top.offer(x > top.least, x, index);
    };
    if (r.first && warp == 0 && r.head > 0) single(lane < r.head, lane);
    for (int turn = 0; turn < r.turns; ++turn) {
#pragma unroll 1
        for (int i = 0; i < kLpLoads; ++i) {
            const int v = r.vector_at(turn, i);
            float x[VEC];
            if (v < r.v_end) {
                unpack_vec<T, VEC>(r.vec[v], x);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) x[j] = -INFINITY;
            }
            // an element equal to the least of a full list comes later in the row than all that are listed, unless
            // it is one of this vector's
            const float over = top.least;
#pragma unroll
            for (int j = 0; j < VEC; ++j) top.offer(x[j] > over, x[j], r.head + v * VEC + j);
        }
    }
    if (r.last && warp == kLpWarps - 1 && r.tail0 < r.vocab) single(r.tail0 + lane < r.vocab, r.tail0 + lane);
    warp_top[warp][lane] = lane < k ? top.key : 0ull;
    if (threadIdx.x < kMaxTop) best[threadIdx.x] = 0ull;
    __syncthreads();
    // an entry's place is the number of larger ones (no two are equal)
    const unsigned long long mine = warp_top[warp][lane];
    int rank = 0;
    for (int w = 0; w < kLpWarps; ++w)
        for (int j = 0; j < k; ++j) rank += warp_top[w][j] > mine ? 1 : 0;
    if (mine != 0ull && rank < k) best[rank] = mine;
    __syncthreads();
}

template <typename T, bool kTop, int kLpLoads>
__global__ void __launch_bounds__(kLpThreads, kLpLoads == kFewRowsLoads ? 2 : 3) logprobs_kernel(const __grid_constant__ LogprobsParams p) {
    constexpr int VEC = RowPart<T, kLpLoads>::VEC;
    constexpr int NB = kLpUnroll * VEC;                 // elements of a thread's block
    __shared__ int warp_tops[kLpWarps];
    __shared__ float2 warp_sums[kLpWarps];
    __shared__ unsigned long long best[kMaxTop];
    // what the row's blocks bring to the first one
    __shared__ __align__(16) Stat all_stat[kMaxCluster];
    __shared__ unsigned long long all_top[kTop ? kMaxCluster : 1][kMaxTop];
    __shared__ __align__(16) float thread_max[kTop ? kLpThreads : 4];
    __shared__ unsigned long long found[kTop ? kFound : 1];
    __shared__ int n_found, floor_of_top;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int part = p.ctas > 1 ? (int)cluster_ctarank() : 0;
    const long long row = blockIdx.x / (unsigned)p.ctas;
    if (p.ctas > 1) cluster_sync_all();                 // every block of the row is there to be written to
    pdl_wait();
    pdl_launch_dependents();
    const RowPart<T, kLpLoads> r(p, row, part);
    // the token asked for and its logit: two loads in a row, well before they are needed
    long long token = -1;
    float token_x = 0.f;
    if (part == 0 && threadIdx.x == 0 && p.tokens) {
        token = p.tokens[row];
        if (token >= 0 && token < p.vocab) token_x = to_f32<T>(r.x[token]);
    }

    Stat st = no_elements();
    auto single = [&](bool have, int index) {           // one element per lane: a row's ragged ends
        const float x = have ? to_f32<T>(r.x[index]) : -INFINITY;
        if (x > st.m) rebase(st, x);
        if (!(x > -INFINITY) && !(x != x)) return;
        const float y = fabsf(st.m) > kFar ? far_y(x, st.m) : fmaf(x, kLog2e, -st.r);
        const float e = ex2(y);
        st.l += e;
        st.u = fmaf(e, fmaxf(y, -200.f), st.u);
    };
    if (r.first && warp == 0 && r.head > 0) single(lane < r.head, lane);
    if (r.last && warp == kLpWarps - 1 && r.tail0 < r.vocab) single(r.tail0 + lane < r.vocab, r.tail0 + lane);

    uint4 cur[kLpLoads];
    auto load = [&](int turn, uint4 (&d)[kLpLoads]) {
        constexpr uint32_t none = Vec16<T>::kNone;
#pragma unroll
        for (int i = 0; i < kLpLoads; ++i) {
            const int v = r.vector_at(turn, i);
            d[i] = make_uint4(none, none, none, none);
            if (v < r.v_end) d[i] = __ldcs(r.vec + v);
        }
    };
    int best_block = -1;                                // where the thread's maximum was (-1: at the ragged ends)
    float other_max = -INFINITY;                        // the largest of its other blocks' maxima
    load(0, cur);
    for (int turn = 0; turn < r.turns; ++turn) {
        uint4 next[kLpLoads];
        load(turn + 1, next);
#pragma unroll
        for (int h = 0; h < kLpLoads; h += kLpUnroll) {
            uint4 raw[kLpUnroll];
#pragma unroll
            for (int i = 0; i < kLpUnroll; ++i) raw[i] = cur[h + i];
            const float bm = Vec16<T>::max_of(raw);
            if (bm > st.m) {
                if (kTop) {
                    other_max = st.m;
                    best_block = turn * (kLpLoads / kLpUnroll) + h / kLpUnroll;
                }
                rebase(st, bm);
            } else if (kTop) {
                other_max = fmaxf(other_max, bm);
            }
            float x[NB];
#pragma unroll
            for (int i = 0; i < kLpUnroll; ++i) unpack_vec<T, VEC>(raw[i], &x[i * VEC]);
            // the block's own sums first: shorter chains of roundings
            float l = 0.f, u = 0.f;
            if (fabsf(st.m) <= kFar || st.m == -INFINITY) {
                const float r0 = st.m == -INFINITY ? 0.f : st.r;
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const float y = fmaf(x[j], kLog2e, -r0), e = ex2(y);
                    l += e;
                    u = fmaf(e, fmaxf(y, -200.f), u);   // (-infinity: weight 0 times a finite number)
                }
            } else {
#pragma unroll 1
                for (int i = 0; i < kLpUnroll; ++i) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float y = far_y(x[j], st.m), e = ex2(y);
                        l += e;
                        u = fmaf(e, fmaxf(y, -200.f), u);
                    }
#pragma unroll
                    for (int j = 0; j + VEC < NB; ++j) x[j] = x[j + VEC];
                }
            }
            st.l += l;
            st.u += u;
        }
#pragma unroll
        for (int i = 0; i < kLpLoads; ++i) cur[i] = next[i];
    }
    if constexpr (kTop) {
        thread_max[threadIdx.x] = st.m;
        if (threadIdx.x < kMaxTop) best[threadIdx.x] = 0ull;
        if (threadIdx.x == 0) n_found = 0;
    }

    // ---- the block's maximum; every thread's sums relative to it, added up
    const float my_max = st.m;
    const int warp_max = __reduce_max_sync(0xffffffffu, ordered_int(st.m));
    if (lane == 0) warp_tops[warp] = warp_max;
    __syncthreads();
    int block_max = warp_tops[0];
#pragma unroll
    for (int w = 1; w < kLpWarps; ++w) block_max = max(block_max, warp_tops[w]);
    rebase(st, from_ordered(block_max));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        st.l += __shfl_xor_sync(0xffffffffu, st.l, o);
        st.u += __shfl_xor_sync(0xffffffffu, st.u, o);
    }
    if (lane == 0) warp_sums[warp] = make_float2(st.l, st.u);
    if constexpr (kTop) {
        // The p.top-th largest of the threads' maxima, to its 16 leading bits and rounded down (a slightly lower floor is
        // one too): two bits at a time, the largest value that as many of them reach.
        if (warp == 0) {
            uint32_t v[kLpWarps], bits = 0u;
#pragma unroll
            for (int i = 0; i < kLpWarps; ++i) v[i] = (uint32_t)ordered_int(thread_max[i * 32 + lane]) ^ 0x80000000u;
#pragma unroll
            for (int b = 30; b >= 16; b -= 2) {
                uint32_t reach = 0u;                    // threads that reach each of the three next values, 10 bits each
#pragma unroll
                for (int i = 0; i < kLpWarps; ++i)
                    reach += (v[i] >= (bits | (1u << b)) ? 1u : 0u) + (v[i] >= (bits | (2u << b)) ? 1u << 10 : 0u) +
                             (v[i] >= (bits | (3u << b)) ? 1u << 20 : 0u);
                reach = __reduce_add_sync(0xffffffffu, reach);
                const uint32_t k = (uint32_t)p.top;
                bits |= (reach >> 20) >= k ? 3u << b : ((reach >> 10) & 1023u) >= k ? 2u << b : (reach & 1023u) >= k ? 1u << b : 0u;
            }
            static_assert(kLpThreads < 1024, "counts of ten bits");
            if (lane == 0) floor_of_top = (int)(bits ^ 0x80000000u);
        }
        __syncthreads();
        const int least_int = floor_of_top;
        auto find = [&](float x, int index) {
            // (the floor of a masked row lies below -infinity, among the NaN)
            if (ordered_int(x) >= least_int && x > -INFINITY) {
                const int at = atomicAdd(&n_found, 1);
                if (at < kFound) found[at] = key_of(x, index);
            }
        };
        if (r.first && warp == 0 && lane < r.head) find(to_f32<T>(r.x[lane]), lane);
        if (r.last && warp == kLpWarps - 1 && r.tail0 + lane < r.vocab) find(to_f32<T>(r.x[r.tail0 + lane]), r.tail0 + lane);
        auto look = [&](int v) {
            if (v >= r.v_end) return;
            float x[VEC];
            unpack_vec<T, VEC>(__ldg(r.vec + v), x);
#pragma unroll
            for (int j = 0; j < VEC; ++j) find(x[j], r.head + v * VEC + j);
        };
        constexpr int kPer = kLpLoads / kLpUnroll;      // blocks per turn
        if (best_block >= 0 && ordered_int(my_max) >= least_int) {
#pragma unroll
            for (int i = 0; i < kLpUnroll; ++i) look(r.vector_at(best_block / kPer, best_block % kPer * kLpUnroll + i));
        }
        // threads of which another block reaches it: the warp reads all of the thread's vectors, one to a lane
        uint32_t todo = __ballot_sync(0xffffffffu, other_max > -INFINITY && ordered_int(other_max) >= least_int);
        // (all lanes go on or stop together)
        while (todo && !__any_sync(0xffffffffu, *(volatile int *)&n_found > kFound)) {
            const int src = __ffs((int)todo) - 1;
            todo &= todo - 1;
            const int done = __shfl_sync(0xffffffffu, best_block, src);
            for (int i = lane; i < r.turns * kLpLoads; i += 32)
                if (i / kLpUnroll != done) look(r.vector_at(i / kLpLoads, i % kLpLoads) + src - lane);
        }
        __syncwarp();
        __syncthreads();
        const int n = n_found;
        if (n <= kFound) {
            // an element's place is the number of larger ones
            for (int i = threadIdx.x; i < n; i += kLpThreads) {
                const unsigned long long mine = found[i];
                int rank = 0;
                for (int j = 0; j < n; ++j) rank += found[j] > mine ? 1 : 0;
                if (rank < p.top) best[rank] = mine;
            }
            __syncthreads();
        } else {
            // (the found elements' memory holds the lists now)
            top_by_lists<T, kLpLoads>(r, p.top, reinterpret_cast<unsigned long long(*)[kMaxTop]>(found), best);
        }
        if (p.ctas > 1 && threadIdx.x < kMaxTop) {
            const uint32_t a = map_to_rank(smem_u32(&all_top[part][threadIdx.x]), 0);
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(a), "l"(best[threadIdx.x]) : "memory");
        }
    }
    if constexpr (!kTop) __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < kLpWarps; ++w) {
            st.l += warp_sums[w].x;
            st.u += warp_sums[w].y;
        }
        st_cluster_v4(map_to_rank(smem_u32(&all_stat[part]), 0), st.m, st.r, st.l, st.u);
    }
    if (p.ctas > 1) {
        cluster_sync_all();                             // the parts are in the first block's shared memory
        if (part != 0) return;
        if constexpr (kTop) {
            const unsigned long long mine = warp < p.ctas ? all_top[warp][lane] : 0ull;
            if (threadIdx.x < kMaxTop) best[threadIdx.x] = 0ull;
            __syncthreads();
            int rank = 0;
            if (lane < p.top)
                for (int w = 0; w < p.ctas; ++w)
                    for (int j = 0; j < p.top; ++j) rank += all_top[w][j] > mine ? 1 : 0;
            if (mine != 0ull && rank < p.top) best[rank] = mine;
            __syncthreads();
        }
    }
    static_assert(kMaxCluster <= kLpWarps && kFound >= kLpWarps * kMaxTop, "one warp per list, and room for the lists");
    if (warp != 0) return;
    __syncwarp();                                       // (all_stat[0] is lane 0's own write)
    Stat s = lane < p.ctas ? all_stat[lane] : no_elements();
    rebase(s, from_ordered(__reduce_max_sync(0xffffffffu, ordered_int(s.m))));
#pragma unroll
    for (int o = kMaxCluster / 2; o > 0; o >>= 1) {
        s.l += __shfl_xor_sync(0xffffffffu, s.l, o);
        s.u += __shfl_xor_sync(0xffffffffu, s.u, o);
    }
    s.l = __shfl_sync(0xffffffffu, s.l, 0);             // (lanes past the blocks hold sums of nothing)
    s.u = __shfl_sync(0xffffffffu, s.u, 0);
    const bool none = s.l == 0.f;                       // no element above -infinity
    const float log_l = none ? 0.f : log2f(s.l);
    const float from = y_offset(s.m) - log_l;
    auto logprob_of = [&](float x) {
        // x - m as it is; ln 2 times the rounding that r holds (see Stat) less the sum's logarithm
        return none ? -INFINITY : (x - s.m) + from * kLn2;
    };
    if (lane == 0) {
        if (p.logprob) {
            float lp = 0.f;
            if (token >= p.vocab) {
                lp = NAN;
                record_op_error(&g_logprobs_error, (int)row, kSiteToken);
            } else if (token >= 0) {
                lp = logprob_of(token_x);
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

template <typename T, bool kTop>
wsm_status run_logprobs(const LogprobsParams &p, int sms, cudaStream_t stream) {
    const long long blocks = (long long)p.rows * p.ctas;
    const dim3 grid((unsigned)blocks);
    return blocks <= 2ll * sms ? op_launch(&logprobs_kernel<T, kTop, kFewRowsLoads>, grid, kLpThreads, 0, stream, p, p.ctas)
                               : op_launch(&logprobs_kernel<T, kTop, kManyRowsLoads>, grid, kLpThreads, 0, stream, p, p.ctas);
}
template <typename T> wsm_status run_logprobs(const LogprobsParams &p, int sms, cudaStream_t stream) {
    return p.top > 0 ? run_logprobs<T, true>(p, sms, stream) : run_logprobs<T, false>(p, sms, stream);
}

}  // namespace

wsm_status logprobs_error_ptr(void **p) {
    WSM_OP_CUDA(cudaGetSymbolAddress(p, g_logprobs_error));
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
    if (a->dtype == WSM_DTYPE_FP32) return run_logprobs<float>(p, sms, stream);
    return a->dtype == WSM_DTYPE_BF16 ? run_logprobs<__nv_bfloat16>(p, sms, stream) : run_logprobs<__half>(p, sms, stream);
}
