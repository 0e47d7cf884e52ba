// wsm_cache.cu -- the paged key-value cache: writing new tokens into it (wsm_paged_cache_append) and the
// attention of one new token of each sequence over it (wsm_paged_attention), the step between the qkv and
// the o projection of a decode step.
#include "wsm_deal.cuh"
#include "wsm_ops.cuh"

#include <algorithm>
#include <cmath>
#include <limits>
#include <type_traits>

namespace wsm {

namespace {

static __device__ unsigned long long g_cache_error;

// ------------------------------------------------------------------ append

struct AppendParams {
    const uint8_t *src[2];          // k and v rows
    uint8_t *dst[2];                // the caches
    long long src_tok[2], src_head[2];              // strides in elements
    long long dst_page[2], dst_tok[2], dst_head[2];
    float scale[2];
    const long long *slots;
    long long n_slots;              // num_pages * page_size
    int page_size, tokens;
    int chunks;                     // 8-element chunks per head
    int per_tok;                    // chunks per token: 2 (k and v) * heads * chunks
    int toks_per_pass;              // tokens a block handles side by side
};

constexpr int kAppendThreads = 256;
constexpr int kAppendUnroll = 4;    // tokens in flight per thread

// Reads a token's keys and values once and writes them once, 16 bytes a thread; nothing to compute but the 8-bit
// rounding.  On a B200: 64 tokens of 8 heads of 128, 2.1 us (a launch; the call costs its host 5.9); 16001 tokens
// 24.1 us, 131 MB at 5.4 TB/s, the floor at copy speed 20.4: a page's rows are 256 bytes in one place each, and two or
// eight tokens' loads in flight instead of four took 25.6 and 30 us.  Into an 8-bit cache 32 us, 98 MB (15.3): a
// division and a rounding to every element come on top, and stores of 8 bytes.
//
// One thread moves the same 8-element chunk (16 bytes) of many tokens: its place within a token is worked
// out once, and kAppendUnroll tokens' loads are in flight before the first store.
template <typename T, bool kE4m3>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(const __grid_constant__ AppendParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int sub = (int)threadIdx.x / p.per_tok;       // which of the pass's tokens (0 when a token fills the block)
    for (int c = (int)threadIdx.x - sub * p.per_tok; c < p.per_tok; c += kAppendThreads) {
        if (sub >= p.toks_per_pass) break;
        const int half = p.per_tok >> 1;
        const int kv = c >= half ? 1 : 0;
        const int r = c - kv * half;
        const int h = r / p.chunks;
        const long long col = (long long)(r - h * p.chunks) * 8;
        const T *src = reinterpret_cast<const T *>(p.src[kv]) + h * p.src_head[kv] + col;
        const long long dst0 = h * p.dst_head[kv] + col;
        const long long step = (long long)gridDim.x * p.toks_per_pass;
        for (long long t0 = (long long)blockIdx.x * p.toks_per_pass + sub; t0 < p.tokens; t0 += step * kAppendUnroll) {
            long long slot[kAppendUnroll];
            uint4 v[kAppendUnroll];
#pragma unroll
            for (int i = 0; i < kAppendUnroll; ++i) {
                const long long t = t0 + i * step;
                slot[i] = t < p.tokens ? p.slots[t] : -1;
            }
#pragma unroll
            for (int i = 0; i < kAppendUnroll; ++i) {
                const long long t = t0 + i * step;
                if (t < p.tokens) v[i] = __ldcs(reinterpret_cast<const uint4 *>(src + t * p.src_tok[kv]));
            }
#pragma unroll
            for (int i = 0; i < kAppendUnroll; ++i) {
                if (slot[i] < 0) continue;              // no place: a padded row
                if (slot[i] >= p.n_slots) {
                    if (c == 0) record_op_error(&g_cache_error, (int)(t0 + i * step), kSiteSlot);
                    continue;
                }
                long long page;
                int off;
                if (p.n_slots <= 0xffffffffll) {        // 64-bit division costs tens of instructions
                    const uint32_t s = (uint32_t)slot[i], q = s / (uint32_t)p.page_size;
                    page = q;
                    off = (int)(s - q * (uint32_t)p.page_size);
                } else {
                    page = slot[i] / p.page_size;
                    off = (int)(slot[i] - page * p.page_size);
                }
                const long long at = page * p.dst_page[kv] + off * p.dst_tok[kv] + dst0;
                if constexpr (kE4m3) {
                    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
                    uint16_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = unpack2<T>(w[j]);
                        // rounded to the nearest 8-bit value; beyond its range the largest one, not NaN
                        o[j] = (uint16_t)__nv_cvt_float2_to_fp8x2(
                            make_float2(__fdiv_rn(f.x, p.scale[kv]), __fdiv_rn(f.y, p.scale[kv])), __NV_SATFINITE,
                            __NV_E4M3);
                    }
                    *reinterpret_cast<uint2 *>(p.dst[kv] + at) =
                        make_uint2((uint32_t)o[0] | ((uint32_t)o[1] << 16), (uint32_t)o[2] | ((uint32_t)o[3] << 16));
                } else {
                    *reinterpret_cast<uint4 *>(reinterpret_cast<T *>(p.dst[kv]) + at) = v[i];
                }
            }
        }
    }
}

// ------------------------------------------------------------------ attention
//
// For a sequence of n tokens, a query head and the keys and values of the head it shares:
//     s_j = scale * k_scale * q . k_j,  m = max s_j,  l = sum e^(s_j - m),
//     o = v_scale / l * sum e^(s_j - m) v_j,  lse = m + ln l
// in one pass over the cache: weights relative to a reference that follows the running maximum, and a sum and
// output that are rescaled when it moves.  Parts of a sequence computed apart have a (reference, sum, output) of
// their own and join exactly by the same rule.
//
// What bounds it is reading the cache once.  So the work is cut by cache bytes, not by sequences: the
// groups of kGroup tokens of all (sequence, key-value head, query tile) items, laid end to end, are dealt
// out in equal consecutive ranges to the warps of a grid that fills the GPU -- one long sequence and a
// ragged batch balance alike.  A warp streams its range through a cp.async ring of its own (no block-wide
// barrier anywhere); the up to 16 query heads that share a key-value head are the rows of the matrix
// instruction, so a key is read once for all of them.  mma.sync, not tcgen05: at 4 to 16 query rows a
// 128-row tensor-memory tile would be nearly empty, and the tensor work is a small part of the time.
// An item cut between warps leaves fp32 partials that attention_join_kernel adds in range order, so results
// do not depend on timing.
//
// Measured on a B200 (floor: the cache's bytes at the 6440 GB/s of a copy): one token over 131041 of a 16-bit cache of
// 8 heads of 128 101 to 107 us (floor 83); 64 ragged sequences of up to 4000 tokens 36 to 42 us (22); 96 over an 8-bit cache
// 53 to 60 us (34): the warps issue in 54 % of the cycles and the cache comes at 4.2 TB/s; one sequence of 37 tokens
// 7.0 us.  About 4.5 us of each is the chain of reads that finds a warp its first tokens (lengths, then the table, then
// keys), 5 to 6 the join's, which reads its items' places as the main kernel left them.  (Every block of the join
// summing the lengths itself is as fast up to 256 sequences, but grows with the square: 4096 sequences of 20 tokens of
// 32 over 8 heads of 128 took 264 us, 145 now; of 130 tokens 505 and 382.)  With the arithmetic taken out
// the three large ones took 98, 39 and 54 us: what is left lies in the load path and these fixed costs.  A join by the
// last block to arrive instead of a second launch: the same on ragged and long batches, 71 us on the 8-bit one, whose
// registers it took.

constexpr int kMaxBatch = 4096;     // sequences per call: their group prefix sums sit in shared memory
// Weights are 2^(score - reference), the reference kBelow under the running maximum: so a weight of 2^-31 of the
// largest is still an fp16 number, and the largest is 2^kBelow but for the rounding of its score, too little for the
// 16 bits to show -- where one token has nearly all the weight, the output is its value.  (A reference that moves only
// when the maximum has left it by far saves most rescalings, 2 % of a call over an 8-bit cache, but rounds the largest
// weight: errors 1.3 times.)
constexpr float kBelow = 7.f;
// The reference comes from a rounded score, the weight's exponent from the unrounded one (one multiply-add).  They
// differ by half a step of the score: 2^-15 up to kFar, but tens from 2^29 on, where a weight would overflow or vanish.
// Past kFar the score is rounded before the reference is taken from it, so the largest weight is a whole power of two
// (2^7, and 2^0 to 2^8 from 2^24 on, where the reference itself is rounded).
constexpr float kFar = 1024.f;

struct AttnParams {
    const uint8_t *Q;
    const uint8_t *K, *V;
    uint8_t *O;
    float *lse;
    const int *table, *lengths;
    float *part_o;                  // [workers][2][16][D]
    float2 *part_ml;                // [workers][2][16]: reference (base 2) and sum
    int *prefix;                    // [batch + 2], for the join (NULL: none follows): the groups before each sequence and
                                    // in all, and the length of a range
    long long q_row, q_head, o_row, o_head;        // elements
    long long k_page, k_tok, k_head, v_page, v_tok, v_head;
    long long table_stride;
    long long num_pages;
    float sl2;                      // |scale| * k_scale * log2(e), not 0
    int negate;                     // the scale is negative
    float v_scale;
    int batch, heads, kv_heads, group, q_tiles;    // group = heads / kv_heads
    int page_size, page_shift, max_tokens, window; // page_shift: log2 of page_size, or -1
    int kv_alike;                   // K and V have the same strides
    int far;                        // some row lies 2^32 or more 16-byte units into its cache
    int workers;
    int rows_per_cta, join_split;   // join: rows of an item one block takes, and the warps for each
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1);
template <>
__device__ __forceinline__ void mma16816<__nv_bfloat16>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <>
__device__ __forceinline__ void mma16816<__half>(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four e4m3 values as fp16, two to a register: exact.
__device__ __forceinline__ void e4m3x4_half2(uint32_t v, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}

// Block geometry of one instantiation: as many warps and ring stages as registers and shared memory hold.
// In flight per SM: warps * stages * 2 * 16 tokens' rows, 120-210 KB.
template <int D, int ESZ> struct AttnGeo {
    static constexpr int kRow = D * ESZ + 16;           // padded: 8 rows of one 16-byte column in 8 bank groups
    static constexpr int kStage = 2 * kGroup * kRow;
    // 4 KB groups want more warps: a warp's own latency per group, about 1500 clocks, bounds 8 of them
    static constexpr int kWarps = D >= 256 ? 4 : D * ESZ <= 128 ? 12 : 8;
    static constexpr int kFit = 206 * 1024 / (kWarps * kStage);
    static constexpr int kStages = kFit > 8 ? 8 : kFit;
    static constexpr int kRing = kWarps * kStages * kStage;
    static_assert(kStages >= 2, "two stages at least");
};

template <typename T, bool kE4m3, int D>
__global__ void __launch_bounds__(AttnGeo<D, kE4m3 ? 1 : 2>::kWarps * 32, 1)
    attention_kernel(const __grid_constant__ AttnParams p) {
    using Geo = AttnGeo<D, kE4m3 ? 1 : 2>;
    // With an 8-bit cache both products run in fp16 whatever the queries' type: every e4m3 value is one, and
    // 16-bit weights of 2^kBelow or so lose less there than in bf16.  A bf16 query row is brought into fp16's range by
    // a power of two, which the score factor takes back: exact but for elements 2^-30 of the row's largest.
    using M = typename std::conditional<kE4m3, __half, T>::type;
    constexpr int ESZ = kE4m3 ? 1 : 2;
    constexpr int NW = Geo::kWarps, NS = Geo::kStages;
    constexpr int CH = D * ESZ / 16;                    // 16-byte chunks per row
    constexpr int KS = D / 16;                          // MMA k-steps over the head dimension
    extern __shared__ __align__(128) uint8_t smem[];
    int *prefix = reinterpret_cast<int *>(smem + Geo::kRing);
    __shared__ int warp_sums[NW];
    __shared__ uint32_t stage_mask[NW][NS];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hq = p.kv_heads * p.q_tiles;              // items per sequence
    pdl_wait();
    pdl_launch_dependents();

    // ---- prefix sums of the sequences' groups (each block its own copy)
    int carry = 0;
    for (int b0 = 0; b0 < p.batch; b0 += NW * 32) {
        const int b = b0 + (int)threadIdx.x;
        int len = b < p.batch ? p.lengths[b] : 0;
        if (blockIdx.x == 0 && len > p.max_tokens) record_op_error(&g_cache_error, b, kSiteLength);
        int v = span_of(p.max_tokens, p.window, len).groups;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += u;
        }
        if (lane == 31) warp_sums[warp] = v;
        __syncthreads();
        int before = carry;
        for (int w = 0; w < NW; ++w) {
            const int s = warp_sums[w];
            if (w < warp) before += s;
            carry += s;
        }
        if (b < p.batch) {
            prefix[b + 1] = before + v;
            if (blockIdx.x == 0 && p.prefix) p.prefix[b + 1] = before + v;
        }
        if (b == 0) {
            prefix[0] = 0;
            if (blockIdx.x == 0 && p.prefix) p.prefix[0] = 0;
        }
        __syncthreads();
    }

    // ---- this warp's range; neighbouring ranges lie on different SMs, so a short call's few spread over the GPU
    const int worker = warp * (int)gridDim.x + (int)blockIdx.x;
    const int total = line_of(prefix, hq, p.batch);
    const int per = share_of(total, p.workers);
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.prefix) p.prefix[p.batch + 1] = per;

    // ---- sequences without a token to attend to: zeros, and the empty sum's logarithm
    for (int b = worker; b < p.batch; b += p.workers) {
        if (prefix[b + 1] != prefix[b]) continue;
        for (int h = 0; h < p.heads; ++h) {
            T *out = reinterpret_cast<T *>(p.O) + b * p.o_row + h * p.o_head;
            for (int d = lane * 8; d < D; d += 256) *reinterpret_cast<uint4 *>(out + d) = make_uint4(0u, 0u, 0u, 0u);
            if (p.lse && lane == 0) p.lse[(long long)b * p.heads + h] = -INFINITY;
        }
    }

    // (odd lanes work out where the next range begins, even ones where this does)
    Place first = place_of(prefix, p.batch, hq, total, per, worker + (lane & 1));
    const int mine = groups_before(prefix, hq, first, p.batch);
    const int n_groups = __shfl_sync(0xffffffffu, mine, 1) - __shfl_sync(0xffffffffu, mine, 0);
    if (n_groups <= 0) return;
    first.b = __shfl_sync(0xffffffffu, first.b, 0);
    first.item = __shfl_sync(0xffffffffu, first.item, 0);
    first.g = __shfl_sync(0xffffffffu, first.g, 0);

    uint8_t *ring = smem + warp * (NS * Geo::kStage);
    const uint32_t ring_u = smem_u32(ring);

    // ---- the load side: where the next group to look up lies
    int lb = first.b, litem = first.item, lg = first.g;
    while (prefix[lb + 1] == prefix[lb]) {              // (the range holds groups, so a sequence that has some follows)
        ++lb;
        litem = lg = 0;
    }
    const Place start = {lb, litem, lg};
    Span ls = span_of(p.max_tokens, p.window, p.lengths[lb]);
    const int start_groups = ls.groups;
    int next_len = lb + 1 < p.batch ? p.lengths[lb + 1] : 0;    // fetched a sequence ahead
    // Two groups at a time, looked up two groups ahead: lanes 0-15 hold the page of the even group's tokens, lanes
    // 16-31 that of the odd one's.
    struct Pages {
        int page, off, seq, head;
        bool in;
    };
    int looked = 0;                                     // groups looked up
    auto look_up = [&]() {
        Pages r;
        r.page = -1;
        r.off = r.seq = r.head = 0;
        r.in = false;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (looked < n_groups) {
                if ((lane >> 4) == half) {
                    const int tok = ls.base + lg * kGroup + (lane & 15);
                    r.in = tok >= ls.first && tok < ls.len;
                    r.seq = lb;
                    r.head = p.q_tiles == 1 ? litem : litem / p.q_tiles;
                    if (r.in) {
                        const int pi = p.page_shift >= 0 ? tok >> p.page_shift : tok / p.page_size;
                        r.off = tok - pi * p.page_size;
                        r.page = p.table[lb * p.table_stride + pi];
                    }
                }
                ++looked;
                // the next group, over sequences without any
                if (++lg == ls.groups) {
                    lg = 0;
                    if (++litem == hq && looked < n_groups) {
                        litem = 0;
                        ++lb;
                        int len = next_len;
                        while (prefix[lb + 1] == prefix[lb]) len = p.lengths[++lb];
                        ls = span_of(p.max_tokens, p.window, len);
                        next_len = lb + 1 < p.batch ? p.lengths[lb + 1] : 0;
                    }
                }
            }
        }
        return r;
    };
    Pages ahead = look_up();
    // of the pair being loaded: which tokens are there, and where their rows lie, in 16-byte units
    uint32_t there = 0u, k_lo = 0u, k_hi = 0u, v_lo = 0u, v_hi = 0u;
    auto load_group = [&](int k, int stage) {
        if ((k & 1) == 0) {
            const Pages now = ahead;
            const bool ok = now.in && (unsigned)now.page < (unsigned)p.num_pages;
            if (now.in && !ok) record_op_error(&g_cache_error, now.seq, kSitePage);
            there = __ballot_sync(0xffffffffu, ok);
            const unsigned long long ko = ok ? (now.page * p.k_page + now.off * p.k_tok + now.head * p.k_head) * ESZ / 16 : 0;
            k_lo = (uint32_t)ko;
            k_hi = (uint32_t)(ko >> 32);
            if (!p.kv_alike) {
                const unsigned long long vo = ok ? (now.page * p.v_page + now.off * p.v_tok + now.head * p.v_head) * ESZ / 16 : 0;
                v_lo = (uint32_t)vo;
                v_hi = (uint32_t)(vo >> 32);
            }
            ahead = look_up();
        }
        const int half = (k & 1) * 16;
        const uint32_t mask = (there >> half) & 0xffffu;
        if (lane == 0) stage_mask[warp][stage] = mask;
        const uint32_t st = ring_u + (uint32_t)(stage * Geo::kStage);
        // consecutive lanes take consecutive 16-byte chunks of a row; rows that are not there read as zeros
#pragma unroll
        for (int i = 0; i < kGroup * CH / 32; ++i) {
            const int idx = i * 32 + lane;
            const int row = idx / CH, ch = idx % CH;
            const uint32_t bytes = ((mask >> row) << 4) & 16u;
            const uint32_t dst = st + (uint32_t)(row * Geo::kRow + ch * 16);
            unsigned long long rk = __shfl_sync(0xffffffffu, k_lo, half + row);
            if (p.far) rk |= (unsigned long long)__shfl_sync(0xffffffffu, k_hi, half + row) << 32;
            unsigned long long rv = rk;
            if (!p.kv_alike) {
                rv = __shfl_sync(0xffffffffu, v_lo, half + row);
                if (p.far) rv |= (unsigned long long)__shfl_sync(0xffffffffu, v_hi, half + row) << 32;
            }
            cp_async16(dst, p.K + rk * 16 + ch * 16, bytes);
            cp_async16(dst + (uint32_t)(kGroup * Geo::kRow), p.V + rv * 16 + ch * 16, bytes);
        }
    };

    // ---- the compute side
    int cb = start.b, cgroups = start_groups, citem = start.item, cg = start.g;
    int seg_begin = 0;                                  // where the current item's part of this range begins
    const int g = lane >> 2, t = lane & 3;
    uint32_t qa[KS][4];
    float o[2 * KS][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f, f0 = 0.f, f1 = 0.f;
    bool far = false;                                   // a reference of the warp's is past kFar
    auto begin_item = [&]() {
        const int h = p.q_tiles == 1 ? citem : citem / p.q_tiles, qt = citem - h * p.q_tiles;
        const int rows = min(16, p.group - qt * 16);
        const T *q = reinterpret_cast<const T *>(p.Q) + cb * p.q_row + (long long)(h * p.group + qt * 16) * p.q_head;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            // the columns of a step: as ldmatrix leaves the keys (16-bit), or four consecutive bytes of an
            // 8-bit key to a thread, which only permutes the sum's terms
            const int c0 = ks * 16 + (kE4m3 ? 4 * t : 2 * t);
            const int c1 = c0 + (kE4m3 ? 2 : 8);
            qa[ks][0] = g < rows ? *reinterpret_cast<const uint32_t *>(q + g * p.q_head + c0) : 0u;
            qa[ks][1] = g + 8 < rows ? *reinterpret_cast<const uint32_t *>(q + (g + 8) * p.q_head + c0) : 0u;
            qa[ks][2] = g < rows ? *reinterpret_cast<const uint32_t *>(q + g * p.q_head + c1) : 0u;
            qa[ks][3] = g + 8 < rows ? *reinterpret_cast<const uint32_t *>(q + (g + 8) * p.q_head + c1) : 0u;
        }
        if (p.negate) {                                 // (a negative scale: the factor stays positive)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int i = 0; i < 4; ++i) qa[ks][i] ^= 0x80008000u;
        }
        f0 = f1 = p.sl2;
        if constexpr (kE4m3 && std::is_same<T, __nv_bfloat16>::value) {
            float a0 = 0.f, a1 = 0.f;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 u = unpack2<T>(qa[ks][2 * i]), w = unpack2<T>(qa[ks][2 * i + 1]);
                    a0 = fmaxf(a0, fmaxf(fabsf(u.x), fabsf(u.y)));
                    a1 = fmaxf(a1, fmaxf(fabsf(w.x), fabsf(w.y)));
                }
#pragma unroll
            for (int x = 1; x < 4; x <<= 1) {
                a0 = fmaxf(a0, __shfl_xor_sync(0xffffffffu, a0, x));
                a1 = fmaxf(a1, __shfl_xor_sync(0xffffffffu, a1, x));
            }
            // largest element to [2^14, 2^15); zeros, infinities and NaN as they are
            const int e0 = (a0 > 0.f && a0 < INFINITY) ? 14 - ilogbf(a0) : 0;
            const int e1 = (a1 > 0.f && a1 < INFINITY) ? 14 - ilogbf(a1) : 0;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 u = unpack2<T>(qa[ks][2 * i]), w = unpack2<T>(qa[ks][2 * i + 1]);
                    qa[ks][2 * i] = pack2<M>(ldexpf(u.x, e0), ldexpf(u.y, e0));
                    qa[ks][2 * i + 1] = pack2<M>(ldexpf(w.x, e1), ldexpf(w.y, e1));
                }
            f0 = fmaxf(ldexpf(p.sl2, -e0), 1e-37f);
            f1 = fmaxf(ldexpf(p.sl2, -e1), 1e-37f);
        }
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
        far = false;
        // the following item's queries into L1 meanwhile (the next heads of this sequence, or the next sequence's)
        const T *qn = citem + 1 < hq ? q + (long long)rows * p.q_head
                                     : reinterpret_cast<const T *>(p.Q) + min(cb + 1, p.batch - 1) * p.q_row;
        const int ahead_rows = min(16, citem + 1 < hq ? p.heads - (h * p.group + qt * 16 + rows) : p.group);
        for (int i = lane; i < ahead_rows * (D / 64); i += 32)
            asm volatile("prefetch.global.L1 [%0];" ::"l"(qn + (i / (D / 64)) * p.q_head + (i % (D / 64)) * 64));
    };
    // the item's last group in this range is done: outputs when the range holds all of it, else a partial
    auto finish_item = [&](int seg_end) {
        const int h = p.q_tiles == 1 ? citem : citem / p.q_tiles, qt = citem - h * p.q_tiles;
        const int rows = min(16, p.group - qt * 16);
#pragma unroll
        for (int x = 1; x < 4; x <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, x);
            l1 += __shfl_xor_sync(0xffffffffu, l1, x);
        }
        if (seg_end - seg_begin == cgroups) {
            const float r0 = l0 == 0.f ? 0.f : p.v_scale / l0, r1 = l1 == 0.f ? 0.f : p.v_scale / l1;
            T *out = reinterpret_cast<T *>(p.O) + cb * p.o_row + (long long)(h * p.group + qt * 16) * p.o_head;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                uint32_t w[4];
                int d0, d1;
                if constexpr (kE4m3) {
                    // tiles 2 ks and 2 ks + 1 hold the even and odd columns
                    w[0] = pack2<T>(o[2 * ks][0] * r0, o[2 * ks + 1][0] * r0);
                    w[1] = pack2<T>(o[2 * ks][1] * r0, o[2 * ks + 1][1] * r0);
                    w[2] = pack2<T>(o[2 * ks][2] * r1, o[2 * ks + 1][2] * r1);
                    w[3] = pack2<T>(o[2 * ks][3] * r1, o[2 * ks + 1][3] * r1);
                    d0 = ks * 16 + 4 * t;
                    d1 = d0 + 2;
                } else {
                    w[0] = pack2<T>(o[2 * ks][0] * r0, o[2 * ks][1] * r0);
                    w[1] = pack2<T>(o[2 * ks + 1][0] * r0, o[2 * ks + 1][1] * r0);
                    w[2] = pack2<T>(o[2 * ks][2] * r1, o[2 * ks][3] * r1);
                    w[3] = pack2<T>(o[2 * ks + 1][2] * r1, o[2 * ks + 1][3] * r1);
                    d0 = ks * 16 + 2 * t;
                    d1 = d0 + 8;
                }
                if (g < rows) {
                    *reinterpret_cast<uint32_t *>(out + g * p.o_head + d0) = w[0];
                    *reinterpret_cast<uint32_t *>(out + g * p.o_head + d1) = w[1];
                }
                if (g + 8 < rows) {
                    *reinterpret_cast<uint32_t *>(out + (g + 8) * p.o_head + d0) = w[2];
                    *reinterpret_cast<uint32_t *>(out + (g + 8) * p.o_head + d1) = w[3];
                }
            }
            if (p.lse && t == 0) {
                float *lse = p.lse + (long long)cb * p.heads + h * p.group + qt * 16;
                // the reference is in base 2; no finite score at all leaves l = 0 and -infinity
                if (g < rows) lse[g] = (l0 == 0.f ? -INFINITY : (m0 + log2f(l0)) * 0.693147180559945309f);
                if (g + 8 < rows) lse[g + 8] = (l1 == 0.f ? -INFINITY : (m1 + log2f(l1)) * 0.693147180559945309f);
            }
            return;
        }
        const int slot = slot_of(worker, per, line_of(prefix, hq, cb) + citem * (cgroups + kItemCost));
        float *po = p.part_o + (size_t)slot * 16 * D;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {               // rows g and g + 8
                const int r = g + 8 * j;
                if (r >= rows) continue;
                if constexpr (kE4m3) {
                    *reinterpret_cast<float4 *>(po + r * D + ks * 16 + 4 * t) = make_float4(
                        o[2 * ks][2 * j], o[2 * ks + 1][2 * j], o[2 * ks][2 * j + 1], o[2 * ks + 1][2 * j + 1]);
                } else {
                    *reinterpret_cast<float2 *>(po + r * D + ks * 16 + 2 * t) = make_float2(o[2 * ks][2 * j], o[2 * ks][2 * j + 1]);
                    *reinterpret_cast<float2 *>(po + r * D + ks * 16 + 2 * t + 8) =
                        make_float2(o[2 * ks + 1][2 * j], o[2 * ks + 1][2 * j + 1]);
                }
            }
        }
        if (t == 0) {
            if (g < rows) p.part_ml[slot * 16 + g] = make_float2(m0, l0);
            if (g + 8 < rows) p.part_ml[slot * 16 + g + 8] = make_float2(m1, l1);
        }
    };

    int loaded = 0;
    for (; loaded < NS - 1 && loaded < n_groups; ++loaded) {
        load_group(loaded, loaded);
        cp_async_commit();
    }
    for (int i = loaded; i < NS - 1; ++i) cp_async_commit();   // empty groups keep the wait's count
    begin_item();
    // lane addresses of ldmatrix within a stage
    const uint32_t k_lane = kE4m3 ? (uint32_t)(((lane & 7) + ((lane >> 3) & 1) * 8) * Geo::kRow + (lane >> 4) * 16)
                                  : (uint32_t)(((lane & 7) + (lane >> 4) * 8) * Geo::kRow + ((lane >> 3) & 1) * 16);
    const uint32_t v_lane =
        (uint32_t)(kGroup * Geo::kRow + ((lane & 7) + ((lane >> 3) & 1) * 8) * Geo::kRow + (lane >> 4) * 16);
    int stage = 0, fill = NS - 1;
    for (int i = 0; i < n_groups; ++i) {
        cp_async_wait<NS - 2>();
        __syncwarp();                                   // the group is in shared memory, and its mask; the stage
                                                        // refilled next has been read by every lane
        if (loaded < n_groups) {
            load_group(loaded, fill);
            ++loaded;
        }
        cp_async_commit();
        if (++fill == NS) fill = 0;

        const uint32_t st = ring_u + (uint32_t)(stage * Geo::kStage);
        const uint32_t mask = stage_mask[warp][stage];
        if (++stage == NS) stage = 0;
        // scores: rows = query heads, columns = the group's tokens; even and odd k-steps in chains of their own
        float s[2][2][4] = {};
#pragma unroll
        for (int ks = 0; ks < KS; ks += (kE4m3 ? 2 : 1)) {
            uint32_t b[4];
            ldsm4(st + k_lane + (uint32_t)(ks * 16 * ESZ), b);
            if constexpr (kE4m3) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t lo, hi;
                    e4m3x4_half2(b[c], lo, hi);
                    mma16816<M>(s[c >> 1][c & 1], qa[ks + (c >> 1)], lo, hi);
                }
            } else {
                mma16816<M>(s[ks & 1][0], qa[ks], b[0], b[1]);
                mma16816<M>(s[ks & 1][1], qa[ks], b[2], b[3]);
            }
        }
        float x0[4], x1[4];                             // row g, row g + 8
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x0[j] = s[0][j >> 1][j & 1] + s[1][j >> 1][j & 1];
            x1[j] = s[0][j >> 1][2 + (j & 1)] + s[1][j >> 1][2 + (j & 1)];
        }
        if (mask != 0xffffu) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = (mask >> ((j >> 1) * 8 + 2 * t + (j & 1))) & 1u;
                x0[j] = in ? x0[j] : -INFINITY;
                x1[j] = in ? x1[j] : -INFINITY;
            }
        }
        float n0 = __fmul_rn(fmaxf(fmaxf(x0[0], x0[1]), fmaxf(x0[2], x0[3])), f0);
        float n1 = __fmul_rn(fmaxf(fmaxf(x1[0], x1[1]), fmaxf(x1[2], x1[3])), f1);
        // (a thread of a row's four sees its own four scores: the vote is over all, the maximum is shared only then)
        if (__any_sync(0xffffffffu, n0 > m0 + kBelow || n1 > m1 + kBelow)) {
#pragma unroll
            for (int x = 1; x < 4; x <<= 1) {
                n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, x));
                n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, x));
            }
            n0 = n0 > m0 + kBelow ? n0 - kBelow : m0;
            n1 = n1 > m1 + kBelow ? n1 - kBelow : m1;
            // (a reference still at -infinity has summed nothing yet)
            const float a0 = n0 == m0 ? 1.f : ex2(m0 - n0), a1 = n1 == m1 ? 1.f : ex2(m1 - n1);
            m0 = n0;
            m1 = n1;
            far = __any_sync(0xffffffffu, (fabsf(m0) > kFar && m0 != -INFINITY) || (fabsf(m1) > kFar && m1 != -INFINITY));
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int d = 0; d < 2 * KS; ++d) {
                o[d][0] *= a0;
                o[d][1] *= a0;
                o[d][2] *= a1;
                o[d][3] *= a1;
            }
        }
        const float z0 = m0 == -INFINITY ? 0.f : m0, z1 = m1 == -INFINITY ? 0.f : m1;
        if (!far) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x0[j] = fmaf(x0[j], f0, -z0);
                x1[j] = fmaf(x1[j], f1, -z1);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x0[j] = __fsub_rn(__fmul_rn(x0[j], f0), z0);
                x1[j] = __fsub_rn(__fmul_rn(x1[j], f1), z1);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x0[j] = ex2(x0[j]);
            x1[j] = ex2(x1[j]);
            l0 += x0[j];
            l1 += x1[j];
        }
        // the weights go into the second product in 16 bits: half a step of bf16 is 2^-8 of a weight, random
        // over the tokens, where the output itself is rounded once by as much
        const uint32_t pa[4] = {pack2<M>(x0[0], x0[1]), pack2<M>(x1[0], x1[1]), pack2<M>(x0[2], x0[3]), pack2<M>(x1[2], x1[3])};
#pragma unroll
        for (int ks = 0; ks < KS; ks += (kE4m3 ? 2 : 1)) {
            uint32_t b[4];
            ldsm4_t(st + v_lane + (uint32_t)(ks * 16 * ESZ), b);
            if constexpr (kE4m3) {
                // a register holds two tokens of two columns: even column to one tile, odd to the next
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t even0, odd0, even1, odd1;
                    e4m3x4_half2(__byte_perm(b[2 * c], 0, 0x3120), even0, odd0);
                    e4m3x4_half2(__byte_perm(b[2 * c + 1], 0, 0x3120), even1, odd1);
                    mma16816<M>(o[2 * (ks + c)], pa, even0, even1);
                    mma16816<M>(o[2 * (ks + c) + 1], pa, odd0, odd1);
                }
            } else {
                mma16816<M>(o[2 * ks], pa, b[0], b[1]);
                mma16816<M>(o[2 * ks + 1], pa, b[2], b[3]);
            }
        }
        // the item or the range ends here
        ++cg;
        if (cg == cgroups || i + 1 == n_groups) {
            finish_item(i + 1);
            if (i + 1 < n_groups) {
                seg_begin = i + 1;
                cg = 0;
                if (++citem == hq) {
                    citem = 0;
                    do {
                        ++cb;
                    } while (prefix[cb + 1] == prefix[cb]);     // (the range goes on, so one with groups follows)
                    cgroups = prefix[cb + 1] - prefix[cb];
                }
                begin_item();
            }
        }
    }
    cp_async_wait<0>();
}

// Join the partials of the items that were cut: block (item, rows).  Each row's partials are dealt to as many
// warps as there are for it (p.join_split), which take every join_split-th in range order, kJoinUnroll at a time;
// the warps' sums are added in warp order: the same result every time.
constexpr int kJoinWarps = 16;      // at most
constexpr int kJoinUnroll = 4;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) attention_join_kernel(const __grid_constant__ AttnParams p) {
    __shared__ float4 sum[kJoinWarps][D / 4];
    __shared__ float2 ml[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hq = p.kv_heads * p.q_tiles;
    const int b = (int)blockIdx.x / hq, item = (int)blockIdx.x - b * hq;
    const int h = p.q_tiles == 1 ? item : item / p.q_tiles, qt = item - h * p.q_tiles;
    const int rows = min(16, p.group - qt * 16);
    // what needs no data, and the parameters, before the wait
    const int split = p.join_split, wr = warp / split, ws = warp - wr * split;
    const int r = (int)blockIdx.y * p.rows_per_cta + wr;
    const bool mine = wr < p.rows_per_cta && r < rows;
    const int *prefix = p.prefix, *of_b = prefix + b, *of_all = prefix + p.batch + 1;
    const float *part_o = p.part_o;
    const float2 *part_ml = p.part_ml;
    asm volatile("" : "+l"(of_b), "+l"(of_all), "+l"(part_o), "+l"(part_ml));
    pdl_wait();                                         // (before any return: who comes next waits for this kernel alone)
    // No trigger for the next launch: it comes when this kernel's blocks are through with the scratch, as that call may be
    // one that waits for nothing (WSM_FLAG_INDEPENDENT) and may write there, the scratch being the caller's again.
    // (through L1: all warps of all blocks read the same few words)
    const int before = of_b[0], n = of_b[1] - before, per = of_all[0];
    if (n <= kSnapGroups) return;                       // never cut
    const int at = (before + kItemCost * b) * hq + item * (n + kItemCost);      // where the item lies in the line
    const Ranges ranges = ranges_of(at, n, per);
    const int w0 = ranges.first, w1 = ranges.last;
    if (w0 == w1) return;                               // one range holds it
    const int slot0 = slot_of(w0, per, at);
    constexpr int NV = (D / 4 + 31) / 32;               // float4 columns per lane
    float m = -INFINITY, l = 0.f;
    float4 acc[NV] = {};
    if (mine) {
        for (int wb = w0 + ws; wb <= w1; wb += split * kJoinUnroll) {
            float2 x[kJoinUnroll];
            float4 v[kJoinUnroll][NV];
#pragma unroll
            for (int u = 0; u < kJoinUnroll; ++u) {
                const int w = wb + u * split;
                const size_t slot = (size_t)(w == w0 ? slot0 : 2 * w) * 16 + r;
                x[u] = w <= w1 ? __ldcg(&part_ml[slot]) : make_float2(-INFINITY, 0.f);
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    v[u][i] = (w <= w1 && i * 32 + lane < D / 4)
                                  ? __ldcg(reinterpret_cast<const float4 *>(part_o + slot * D) + i * 32 + lane)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            float mn = m;
#pragma unroll
            for (int u = 0; u < kJoinUnroll; ++u) mn = fmaxf(mn, x[u].x);
            const float z = mn == -INFINITY ? 0.f : mn, a = ex2(m - z);
            m = mn;
            l *= a;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                acc[i].x *= a;
                acc[i].y *= a;
                acc[i].z *= a;
                acc[i].w *= a;
            }
#pragma unroll
            for (int u = 0; u < kJoinUnroll; ++u) {
                const float c = ex2(x[u].x - z);
                l += x[u].y * c;
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    acc[i].x += v[u][i].x * c;
                    acc[i].y += v[u][i].y * c;
                    acc[i].z += v[u][i].z * c;
                    acc[i].w += v[u][i].w * c;
                }
            }
        }
    }
    if (split > 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (i * 32 + lane < D / 4) sum[warp][i * 32 + lane] = acc[i];
        if (lane == 0) ml[warp] = make_float2(m, l);
        __syncthreads();
        if (!mine || ws != 0) return;
        for (int w = 1; w < split; ++w) m = fmaxf(m, ml[warp + w].x);
        const float z = m == -INFINITY ? 0.f : m;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int w = 0; w < split; ++w) {
            const float c = ex2(ml[warp + w].x - z);
            l += ml[warp + w].y * c;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (i * 32 + lane >= D / 4) continue;
                const float4 v = sum[warp + w][i * 32 + lane];
                acc[i].x += v.x * c;
                acc[i].y += v.y * c;
                acc[i].z += v.z * c;
                acc[i].w += v.w * c;
            }
        }
    }
    if (!mine) return;
    const float f = l == 0.f ? 0.f : p.v_scale / l;
    T *out = reinterpret_cast<T *>(p.O) + b * p.o_row + (long long)(h * p.group + qt * 16 + r) * p.o_head;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (i * 32 + lane < D / 4)
            *reinterpret_cast<uint2 *>(out + 4 * (i * 32 + lane)) =
                make_uint2(pack2<T>(acc[i].x * f, acc[i].y * f), pack2<T>(acc[i].z * f, acc[i].w * f));
    if (p.lse && lane == 0)
        p.lse[(long long)b * p.heads + h * p.group + qt * 16 + r] =
            l == 0.f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

// ------------------------------------------------------------------ host side

// A stride between n things: with one there is no step to take, and whatever its stride says is not looked at.
bool stride_ok(long long s, long long n, int vec) { return n <= 1 || (s >= 0 && s % vec == 0); }
long long step_of(long long s, long long n) { return n <= 1 ? 0 : s; }

wsm_status check_cache(const wsm_kv_cache *c) {
    if (!c) return op_fail(WSM_ERR_INVALID, "cache must be non-null");
    if (!c->K || !c->V) return op_fail(WSM_ERR_INVALID, "the cache's K and V must be non-null device pointers");
    if (c->num_pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->head_dim < 1)
        return op_fail(WSM_ERR_INVALID, "the cache needs pages, tokens in a page, heads and a head dimension (got %lld, %d, %d, %d)",
                       c->num_pages, c->page_size, c->kv_heads, c->head_dim);
    if (c->dtype != WSM_DTYPE_BF16 && c->dtype != WSM_DTYPE_FP16 && c->dtype != WSM_DTYPE_E4M3)
        return op_fail(WSM_ERR_UNSUPPORTED, "cache element type %d: bf16, fp16 and e4m3 are", c->dtype);
    if (c->num_pages > (1ll << 31) - 1 || c->num_pages > ((1ll << 62) / c->page_size))
        return op_fail(WSM_ERR_UNSUPPORTED, "%lld pages of %d tokens are too many", c->num_pages, c->page_size);
    const int vec = c->dtype == WSM_DTYPE_E4M3 ? 16 : 8;  // elements in 16 bytes
    if (c->head_dim % vec) return op_fail(WSM_ERR_UNSUPPORTED, "head dimension %d is not a multiple of %d", c->head_dim, vec);
    if (!aligned_to(c->K, 16) || !aligned_to(c->V, 16)) return op_fail(WSM_ERR_ALIGN, "the caches must be 16-byte aligned");
    const long long n[3] = {c->num_pages, c->page_size, c->kv_heads};
    for (int i = 0; i < 3; ++i)
        if (!stride_ok(c->k_strides[i], n[i], vec) || !stride_ok(c->v_strides[i], n[i], vec))
            return op_fail(WSM_ERR_ALIGN, "the cache strides must be multiples of 16 bytes, and not negative");
    if (!(c->k_scale > 0.f) || !(c->v_scale > 0.f) || !(c->k_scale < INFINITY) || !(c->v_scale < INFINITY))
        return op_fail(WSM_ERR_INVALID, "the cache scales must be positive and finite");
    if (c->dtype != WSM_DTYPE_E4M3 && (c->k_scale != 1.f || c->v_scale != 1.f))
        return op_fail(WSM_ERR_INVALID, "a 16-bit cache has scales of 1");
    return WSM_OK;
}

template <typename T, bool kE4m3, int D>
wsm_status run_attention(const AttnParams &p, int dev, int sms, cudaStream_t stream, bool join, dim3 join_grid) {
    using Geo = AttnGeo<D, kE4m3 ? 1 : 2>;
    static volatile bool done[kMaxOpDevices] = {};
    wsm_status st;
    const size_t smem = (size_t)Geo::kRing + (size_t)(p.batch + 1) * 4;
    if ((st = op_allow_smem(&attention_kernel<T, kE4m3, D>, Geo::kRing + (kMaxBatch + 1) * 4, dev, done)) != WSM_OK) return st;
    if ((st = op_launch(&attention_kernel<T, kE4m3, D>, dim3((unsigned)sms), Geo::kWarps * 32, smem, stream, p)) != WSM_OK)
        return st;
    if (!join) return WSM_OK;
    return op_launch(&attention_join_kernel<T, D>, join_grid, p.rows_per_cta * p.join_split * 32, 0, stream, p);
}

int attention_warps(int head_dim, bool e4m3) {
    switch (head_dim) {
        case 64: return e4m3 ? AttnGeo<64, 1>::kWarps : AttnGeo<64, 2>::kWarps;
        case 96: return e4m3 ? AttnGeo<96, 1>::kWarps : AttnGeo<96, 2>::kWarps;
        case 128: return e4m3 ? AttnGeo<128, 1>::kWarps : AttnGeo<128, 2>::kWarps;
        default: return e4m3 ? AttnGeo<256, 1>::kWarps : AttnGeo<256, 2>::kWarps;
    }
}

// No item can be cut when none can have more than kSnapGroups groups.
bool attention_may_cut(long long max_tokens, int window) {
    const long long span = window > 0 ? std::min<long long>(max_tokens, (long long)window + kGroup - 1) : max_tokens;
    return (span + kGroup - 1) / kGroup > kSnapGroups;
}

// Partials of two items per range (the first and the last it holds a part of), and the sequences' places in the line.
size_t attention_ws(int head_dim, bool e4m3, int sms) {
    const size_t slots = (size_t)sms * attention_warps(head_dim, e4m3) * 2;
    return slots * 16 * (size_t)head_dim * 4 + slots * 16 * 8 + (kMaxBatch + 2) * sizeof(int);
}

bool attention_dim_ok(int d) { return d == 64 || d == 96 || d == 128 || d == 256; }

}  // namespace

wsm_status cache_error_ptr(void **p) {
    WSM_OP_CUDA(cudaGetSymbolAddress(p, g_cache_error));
    return WSM_OK;
}

}  // namespace wsm

using namespace wsm;

extern "C" {

wsm_status wsm_paged_cache_append(const wsm_kv_cache *cache, const wsm_kv_rows *rows, wsm_stream_t stream_) {
    wsm_status st = check_cache(cache);
    if (st != WSM_OK) return st;
    if (!rows) return op_fail(WSM_ERR_INVALID, "rows must be non-null");
    if (rows->tokens < 0) return op_fail(WSM_ERR_INVALID, "tokens must not be negative (got %d)", rows->tokens);
    if (rows->dtype != WSM_DTYPE_BF16 && rows->dtype != WSM_DTYPE_FP16)
        return op_fail(WSM_ERR_UNSUPPORTED, "row element type %d: bf16 and fp16 are", rows->dtype);
    if (cache->dtype != WSM_DTYPE_E4M3 && cache->dtype != rows->dtype)
        return op_fail(WSM_ERR_INVALID, "a 16-bit cache takes rows of its own type");
    if (rows->tokens == 0) return WSM_OK;
    if (!rows->k || !rows->v || !rows->slots) return op_fail(WSM_ERR_INVALID, "k, v and slots must be non-null device pointers");
    if (!aligned_to(rows->k, 16) || !aligned_to(rows->v, 16)) return op_fail(WSM_ERR_ALIGN, "k and v must be 16-byte aligned");
    if (!aligned_to(rows->slots, 8)) return op_fail(WSM_ERR_ALIGN, "slots must be 8-byte aligned");
    const long long n_src[2] = {rows->tokens, cache->kv_heads}, n_dst[3] = {cache->num_pages, cache->page_size, cache->kv_heads};
    for (int i = 0; i < 2; ++i)
        if (!stride_ok(rows->k_strides[i], n_src[i], 8) || !stride_ok(rows->v_strides[i], n_src[i], 8))
            return op_fail(WSM_ERR_ALIGN, "the strides of k and v must be multiples of 16 bytes, and not negative");
    for (int i = 0; i < 3; ++i)
        if (n_dst[i] > 1 && (cache->k_strides[i] < cache->head_dim || cache->v_strides[i] < cache->head_dim))
            return op_fail(WSM_ERR_INVALID, "rows of the cache overlap (a stride is below the head dimension)");
    const long long per_tok = 2ll * cache->kv_heads * (cache->head_dim / 8);
    if (per_tok > (1 << 30)) return op_fail(WSM_ERR_UNSUPPORTED, "rows of %d heads of %d are too long", cache->kv_heads, cache->head_dim);
    int dev, sms;
    if ((st = device_sms(&dev, &sms)) != WSM_OK) return st;
    AppendParams p = {};
    p.src[0] = static_cast<const uint8_t *>(rows->k);
    p.src[1] = static_cast<const uint8_t *>(rows->v);
    p.dst[0] = static_cast<uint8_t *>(cache->K);
    p.dst[1] = static_cast<uint8_t *>(cache->V);
    for (int i = 0; i < 2; ++i) {
        const long long *src = i ? rows->v_strides : rows->k_strides;
        const long long *dst = i ? cache->v_strides : cache->k_strides;
        p.src_tok[i] = step_of(src[0], n_src[0]);
        p.src_head[i] = step_of(src[1], n_src[1]);
        p.dst_page[i] = step_of(dst[0], n_dst[0]);
        p.dst_tok[i] = step_of(dst[1], n_dst[1]);
        p.dst_head[i] = step_of(dst[2], n_dst[2]);
    }
    p.scale[0] = cache->k_scale;
    p.scale[1] = cache->v_scale;
    p.slots = rows->slots;
    p.n_slots = cache->num_pages * cache->page_size;
    p.page_size = cache->page_size;
    p.tokens = rows->tokens;
    p.chunks = cache->head_dim / 8;
    p.per_tok = (int)per_tok;
    p.toks_per_pass = std::max(1, kAppendThreads / p.per_tok);
    // blocks for a token (or a pass of small ones) each, up to eight to an SM
    const long long passes = ((long long)p.tokens + p.toks_per_pass - 1) / p.toks_per_pass;
    const dim3 grid((unsigned)std::min<long long>(passes, 8ll * sms));
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    if (cache->dtype == WSM_DTYPE_E4M3)
        return rows->dtype == WSM_DTYPE_BF16 ? op_launch(&append_kernel<__nv_bfloat16, true>, grid, kAppendThreads, 0, stream, p)
                                             : op_launch(&append_kernel<__half, true>, grid, kAppendThreads, 0, stream, p);
    return op_launch(&append_kernel<__half, false>, grid, kAppendThreads, 0, stream, p);  // a copy: any 16-bit type
}

wsm_status wsm_paged_attention_workspace(int batch, int head_dim, int cache_dtype, long long max_tokens, int window,
                                         size_t *bytes) {
    if (!bytes) return op_fail(WSM_ERR_INVALID, "bytes must be non-null");
    if (batch < 0 || max_tokens < 0 || window < 0) return op_fail(WSM_ERR_INVALID, "sizes must not be negative");
    if (batch > kMaxBatch || !attention_dim_ok(head_dim))
        return op_fail(WSM_ERR_UNSUPPORTED, "paged attention takes up to %d sequences and head dimensions 64, 96, 128 and 256 (got %d, %d)",
                       kMaxBatch, batch, head_dim);
    *bytes = 0;
    if (batch == 0 || !attention_may_cut(max_tokens, window)) return WSM_OK;
    int dev, sms;
    wsm_status st = device_sms(&dev, &sms);
    if (st == WSM_OK) *bytes = attention_ws(head_dim, cache_dtype == WSM_DTYPE_E4M3, sms);
    return st;
}

wsm_status wsm_paged_attention(const wsm_kv_cache *cache, const wsm_attention *a, wsm_stream_t stream_) {
    wsm_status st = check_cache(cache);
    if (st != WSM_OK) return st;
    if (!a) return op_fail(WSM_ERR_INVALID, "the attention arguments must be non-null");
    if (a->batch < 0 || a->heads < 1 || a->max_pages < 0 || a->window < 0)
        return op_fail(WSM_ERR_INVALID, "batch %d, heads %d, max_pages %d, window %d: no negative sizes, and a head at least", a->batch,
                       a->heads, a->max_pages, a->window);
    if (a->dtype != WSM_DTYPE_BF16 && a->dtype != WSM_DTYPE_FP16)
        return op_fail(WSM_ERR_UNSUPPORTED, "query element type %d: bf16 and fp16 are", a->dtype);
    if (cache->dtype != WSM_DTYPE_E4M3 && cache->dtype != a->dtype)
        return op_fail(WSM_ERR_INVALID, "a 16-bit cache takes queries of its own type");
    if (!attention_dim_ok(cache->head_dim))
        return op_fail(WSM_ERR_UNSUPPORTED, "head dimension %d: 64, 96, 128 and 256 are", cache->head_dim);
    if (a->heads > 65536) return op_fail(WSM_ERR_UNSUPPORTED, "%d heads: up to 65536 are", a->heads);
    if (a->heads % cache->kv_heads)
        return op_fail(WSM_ERR_INVALID, "%d query heads are not a multiple of %d key-value heads", a->heads, cache->kv_heads);
    if (a->batch > kMaxBatch) return op_fail(WSM_ERR_UNSUPPORTED, "%d sequences: up to %d are", a->batch, kMaxBatch);
    const long long max_tokens = (long long)a->max_pages * cache->page_size;
    if (max_tokens > 0x7fffffffll - kGroup || (max_tokens / kGroup + 1 + kItemCost) * std::max(a->batch, 1) * ((long long)cache->kv_heads * ((a->heads / cache->kv_heads + 15) / 16)) > 0x7fffffffll)
        return op_fail(WSM_ERR_UNSUPPORTED, "%d sequences of up to %lld tokens are too many", a->batch, max_tokens);
    if (!(a->scale > -INFINITY) || !(a->scale < INFINITY)) return op_fail(WSM_ERR_INVALID, "the scale must be finite");
    const double factor = std::fabs((double)a->scale) * cache->k_scale * 1.44269504088896340736;   // of scores in base 2
    if (factor > std::numeric_limits<float>::max())
        return op_fail(WSM_ERR_INVALID, "the scale times the keys' scale, in base 2, is past fp32's range");
    if (a->batch == 0) return WSM_OK;
    const bool e8 = cache->dtype == WSM_DTYPE_E4M3;
    const bool join = attention_may_cut(max_tokens, a->window);
    if (!a->Q || !a->O || !a->lengths || (!a->block_table && a->max_pages > 0) || (!a->workspace && join))
        return op_fail(WSM_ERR_INVALID, "Q, O, lengths, block_table and workspace must be non-null device pointers");
    if (!aligned_to(a->Q, 16) || !aligned_to(a->O, 16) || !aligned_to(a->workspace, 16))
        return op_fail(WSM_ERR_ALIGN, "Q, O and workspace must be 16-byte aligned");
    if (!aligned_to(a->lengths, 4) || !aligned_to(a->block_table, 4) || !aligned_to(a->lse, 4))
        return op_fail(WSM_ERR_ALIGN, "lengths, block_table and lse must be 4-byte aligned");
    const long long n_q[2] = {a->batch, a->heads}, n_c[3] = {cache->num_pages, cache->page_size, cache->kv_heads};
    for (int i = 0; i < 2; ++i) {
        if (!stride_ok(a->q_strides[i], n_q[i], 8) || !stride_ok(a->o_strides[i], n_q[i], 8))
            return op_fail(WSM_ERR_ALIGN, "the strides of Q and O must be multiples of 16 bytes, and not negative");
        if (n_q[i] > 1 && a->o_strides[i] < cache->head_dim)
            return op_fail(WSM_ERR_INVALID, "rows of O overlap (a stride is below the head dimension)");
    }
    if (a->batch > 1 && a->table_stride < 0) return op_fail(WSM_ERR_INVALID, "the table stride must not be negative");
    int dev, sms;
    if ((st = device_sms(&dev, &sms)) != WSM_OK) return st;
    const size_t need = join ? attention_ws(cache->head_dim, e8, sms) : 0;
    if (a->workspace_bytes < need)
        return op_fail(WSM_ERR_NOMEM, "workspace of %zu bytes is smaller than the %zu needed", a->workspace_bytes, need);

    const int D = cache->head_dim;
    AttnParams p = {};
    p.Q = static_cast<const uint8_t *>(a->Q);
    p.K = static_cast<const uint8_t *>(cache->K);
    p.V = static_cast<const uint8_t *>(cache->V);
    p.O = static_cast<uint8_t *>(a->O);
    p.lse = a->lse;
    p.table = a->block_table;
    p.lengths = a->lengths;
    p.workers = sms * attention_warps(D, e8);
    if (join) {
        const size_t slots = (size_t)p.workers * 2;
        p.part_o = static_cast<float *>(a->workspace);
        p.part_ml = reinterpret_cast<float2 *>(p.part_o + slots * 16 * (size_t)D);
        p.prefix = reinterpret_cast<int *>(p.part_ml + slots * 16);
    }
    p.q_row = step_of(a->q_strides[0], n_q[0]);
    p.q_head = step_of(a->q_strides[1], n_q[1]);
    p.o_row = step_of(a->o_strides[0], n_q[0]);
    p.o_head = step_of(a->o_strides[1], n_q[1]);
    p.k_page = step_of(cache->k_strides[0], n_c[0]);
    p.k_tok = step_of(cache->k_strides[1], n_c[1]);
    p.k_head = step_of(cache->k_strides[2], n_c[2]);
    p.v_page = step_of(cache->v_strides[0], n_c[0]);
    p.v_tok = step_of(cache->v_strides[1], n_c[1]);
    p.v_head = step_of(cache->v_strides[2], n_c[2]);
    p.table_stride = step_of(a->table_stride, a->batch);
    p.num_pages = cache->num_pages;
    // (a factor of 0 would make NaN of what is masked; fp32 scores times the least number above it all vanish)
    p.sl2 = std::max((float)factor, std::numeric_limits<float>::denorm_min());
    p.negate = a->scale < 0.f;
    p.v_scale = cache->v_scale;
    p.batch = a->batch;
    p.heads = a->heads;
    p.kv_heads = cache->kv_heads;
    p.group = a->heads / cache->kv_heads;
    p.q_tiles = (p.group + 15) / 16;
    p.page_size = cache->page_size;
    p.page_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (cache->page_size == (1 << i)) p.page_shift = i;
    const double reach = std::max(((double)cache->num_pages - 1) * p.k_page + ((double)cache->page_size - 1) * p.k_tok +
                                      ((double)cache->kv_heads - 1) * p.k_head,
                                  ((double)cache->num_pages - 1) * p.v_page + ((double)cache->page_size - 1) * p.v_tok +
                                      ((double)cache->kv_heads - 1) * p.v_head);
    p.far = reach * (e8 ? 1 : 2) / 16 >= 4294967295.0;
    p.kv_alike = p.k_page == p.v_page && p.k_tok == p.v_tok && p.k_head == p.v_head;
    p.max_tokens = (int)max_tokens;
    p.window = a->window;
    const long long items = (long long)p.batch * p.kv_heads * p.q_tiles;
    if (items > 0x7fffffffll) return op_fail(WSM_ERR_UNSUPPORTED, "%lld items are too many", items);
    const int rows = std::min(16, p.group);
    // a block for each row while there are few (and may be many partials), else one for all of an item's
    p.rows_per_cta = items * rows <= 2ll * sms ? 1 : rows;
    // a warp to a row for every two partials that an item has on average, four to a block at least (on a B200: 512
    // sequences of 4 x 4 heads 68.7 us, 74.6 with sixteen warps to every block; 32 of 32 heads of 64 66.5 and 71.4)
    const int cuts = (int)std::min<long long>(p.workers / items + 2, 1 << 20);
    p.join_split = std::min(std::max((cuts + 1) / 2, (4 + p.rows_per_cta - 1) / p.rows_per_cta), kJoinWarps / p.rows_per_cta);
    const dim3 jg((unsigned)items, (unsigned)((rows + p.rows_per_cta - 1) / p.rows_per_cta));
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const bool bf = a->dtype == WSM_DTYPE_BF16;
#define WSM_ATTN(DIM)                                                                                             \
    case DIM:                                                                                                     \
        if (e8)                                                                                                   \
            return bf ? run_attention<__nv_bfloat16, true, DIM>(p, dev, sms, stream, join, jg)                    \
                      : run_attention<__half, true, DIM>(p, dev, sms, stream, join, jg);                          \
        return bf ? run_attention<__nv_bfloat16, false, DIM>(p, dev, sms, stream, join, jg)                       \
                  : run_attention<__half, false, DIM>(p, dev, sms, stream, join, jg)
    switch (D) {
        WSM_ATTN(64);
        WSM_ATTN(96);
        WSM_ATTN(128);
        WSM_ATTN(256);
    }
#undef WSM_ATTN
    return op_fail(WSM_ERR_UNSUPPORTED, "head dimension %d", D);
}

}  // extern "C"
