// wsm_experts.cu -- matrix products grouped by expert with ragged row counts (wsm_expert_gemm): the gate+up
// and down projections of a mixture-of-experts layer, for one token to whole prompts.
//
//     Y[r, n] = scale_r * sum_k X[r, k] * W[e, n, k]      for the rows r of expert e
//
// What bounds it: with few rows to an expert, reading the weights of the experts that have any (2 N K bytes
// against 2 m N K operations: under about 250 rows each); with more, the tensor cores.  Both want the same
// layout, the product transposed: 128 rows of W are the MMA's M side and an expert's rows its N side, which may
// be any multiple of 16 up to 256, so a handful of rows wastes little and a prompt's fill the instruction.
//
//   experts_plan_kernel (one block) reads the offsets, cuts every expert's product into tiles of 128 weight
//   rows x up to 256 rows of X (an expert's rows cut evenly), and few or last tiles along K into units; it
//   clears the claim and arrival counters of this call.  So nothing outlives a call and nothing needs to have
//   been cleared before.
//   experts_kernel (persistent, one CTA per SM) claims units in order -- SMs do not stream at one rate -- and
//   runs them: warp 0 loads by TMA into a ring of four 48 KB stages, warp 1 issues tcgen05.mma into one of two
//   accumulators in tensor memory, warps 2-9 take finished ones out: activation, scale, rounding, stores.  A
//   tile cut along K leaves fp32 partials, which its last unit to finish adds in K order, so results do not
//   depend on which SM ran what.
//
// Measured on a B200 (floors: weights at the 6440 GB/s of a copy, products at cuBLAS' 1.67 PFLOP/s, 1.39 sustained): 16
// rows over 32 experts of 4096 x 4096, 62 to 71 us by which experts get them (66: weights at 5.6 to 6.2 TB/s, the
// tensor pipe 4 % busy); 1000 rows over 64 experts of 4096 x 1280, 101 to 109 us (106 were all to get rows); 8192 rows
// over 16 experts of 6144 x 4096, 360 to 395 us in a burst and 410 to 480 in a loop, where the power leaves 1.3 to 1.4
// GHz (246, 296), with the tensor pipe 61 % busy.  There some 43 KB a stage come out of L2 at 60 bytes a clock, about what an SM takes in: 550 thousand clocks,
// as many without the products, and 370 without the copies.  CTA pairs (cta_group::2) load 30 % less and took 8 %
// less time there, but as much or 4 % more at 3000 to 8192 rows over smaller experts and 117 to 128 us on the 1000
// rows: half as many tiles are in flight.
#include "wsm_ops.cuh"
#include "wsm_tcgen05.cuh"

#include <algorithm>

namespace wsm {

namespace {

static __device__ int g_experts_status[kOpStatusInts];     // waits that ran out
static __device__ unsigned long long g_experts_error;

constexpr int kMaxExperts = 1024;
constexpr int kTileN = 128;         // weight rows per tile (MMA M)
constexpr int kTileRowsLog = 8;
constexpr int kTileRows = 1 << kTileRowsLog;    // most rows of X per tile (MMA N)
constexpr int kBK = 64;             // K elements per box (a 128-byte swizzle row)
constexpr int kStageBytes = 48 * 1024;
constexpr int kStages = 4;
constexpr int kBoxW = kTileN * kBK * 2;
constexpr int kNarrow = 64;         // up to this many rows a stage holds two K boxes, above one
constexpr int kNarrowX = kNarrow * kBK * 2;
constexpr int kXMaps = 13;          // boxes of 1, 2, 4, 8, 16 and 32, 64, 96 ... 256 rows
// Units announced: the one that the producer writes, one to each of the four stages before it, and the two whose
// accumulators may not have been read.
constexpr int kUnitRing = 8;
constexpr int kEpiSets = 2;
constexpr int kExThreads = 64 + kEpiSets * 128;
constexpr uint32_t kExTmemCols = 2 * kTileRows;
constexpr int kLead = 2;            // a CTA claims its next unit this many stages before its unit ends
constexpr unsigned long long kExWaitNs = 4000000000ull;

// One expert's part of the plan.
struct ExpertRec {
    int lo, m;                      // its rows
    int tile0, unit0;               // tiles and units of the experts before it
    int part0;                      // its first partial, in blocks of 16 rows x 128
    int nu, ku;                     // units of each split tile, K boxes of a unit
    int mrows;                      // rows per tile, a multiple of 16
};
// Head of the scratch: [0] units, [1] tiles before the split ones, [2] claim counter, [3] log2 of a tile's most rows.
enum : int { kHdrUnits = 0, kHdrHead = 1, kHdrClaim = 2, kHdrRowsLog = 3 };
constexpr int kHdrBytes = 256;

struct ExpertParams {
    CUtensorMap tmW;                // [experts][N][K], box 128 x 64
    CUtensorMap tmX[kXMaps];        // [rows][K], boxes box_rows(i) x 64
    void *Y;
    const int *offsets;
    const float *row_scale;
    long long y_stride;
    int *hdr;
    ExpertRec *rec;                 // [experts + 1]
    unsigned int *tile_cnt;         // arrival counters of the split tiles
    float *part;
    int part_cap;                   // partial blocks there is room for
    int cnt_cap;
    int rows, experts, N, K;
    int kb;                         // K boxes
    int n_g;                        // tiles along N
    int silu;
    int sms;
    uint32_t idesc;                 // MMA descriptor without its N
    unsigned long long stall_ns;
};

__host__ __device__ inline int ceil_div(int a, int b) { return (a + b - 1) / b; }

// The box that holds `rows` rows of X, and its height.  One box to a tile: each copy costs the producer thread
// about as much as the next (8192 rows over 16 experts on a B200: 507 us with a tile's rows in two to four boxes,
// 450 us in one), and rows beyond the tile's cost no more than their bytes.
__host__ __device__ inline int box_of(int rows) {
    int i = 0;
    while (i < 4 && (1 << i) < rows) ++i;
    return rows <= 16 ? i : 4 + (rows + 31) / 32;
}
__host__ __device__ inline int box_rows(int i) { return i < 5 ? 1 << i : (i - 4) * 32; }

// Tiles along an expert's rows (cut evenly, a multiple of 16 each).
__device__ __forceinline__ int m_tiles_of(int m, int rows_log) { return (m + (1 << rows_log) - 1) >> rows_log; }

// ------------------------------------------------------------------ plan

template <bool kMax> __device__ __forceinline__ int block_scan(int v, int *warp_tot) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (int)blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = kMax ? max(v, u) : v + u;
    }
    __syncthreads();                                    // (the array may still be read from the scan before)
    if (lane == 31) warp_tot[warp] = v;
    __syncthreads();
    int before = 0;
    for (int w = 0; w < warps; ++w)
        if (w < warp) before = kMax ? max(before, warp_tot[w]) : before + warp_tot[w];
    return kMax ? max(before, v) : before + v;
}

__global__ void __launch_bounds__(kMaxExperts) experts_plan_kernel(const __grid_constant__ ExpertParams p) {
    __shared__ int warp_tot[32];
    __shared__ int tiles_all;
    const int e = threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    for (int i = e; i < p.cnt_cap; i += blockDim.x) p.tile_cnt[i] = 0u;
    // offsets: into [0, rows], never falling
    const bool have = e < p.experts;
    const int raw0 = p.offsets[0];
    const int raw = have ? p.offsets[e + 1] : 0;
    const int lo0 = min(max(raw0, 0), p.rows);
    const int top = have ? min(max(raw, lo0), p.rows) : 0;
    const int hi = max(block_scan<true>(top, warp_tot), lo0);
    int lo = __shfl_up_sync(0xffffffffu, hi, 1);
    if ((e & 31) == 0) {
        lo = lo0;
        for (int w = 0; w < (e >> 5); ++w) lo = max(lo, warp_tot[w]);
    }
    if (have && (raw != hi || (e == 0 && raw0 != lo0))) record_op_error(&g_experts_error, e, kSiteOffsets);
    const int m = have ? hi - lo : 0;
    // The highest tiles read the least (for 256 rows of X 48 KB to a K box, for 64 24 KB), but a call with few of them
    // leaves SMs without: below one to three SMs, lower ones.  (On a B200, 400 rows of 4 experts of 1152 x 3944: 27.8
    // us in tiles of up to 256 rows, 25.6 of 128; 1652 of 15 experts of 304 x 904: 16.5 and 14.6; 300 rows of one expert of
    // 4096 x 4096, 64 tiles, stay with 256: 27 us.)
    int rows_log = kTileRowsLog, mt, tiles, tile_end, total;
    for (;; --rows_log) {
        mt = m_tiles_of(m, rows_log);
        tiles = mt * p.n_g;
        tile_end = block_scan<false>(tiles, warp_tot);
        if (e == (int)blockDim.x - 1) tiles_all = tile_end;
        __syncthreads();
        total = tiles_all;
        if (total >= p.sms / 3 || (1 << rows_log) <= kNarrow) break;
        __syncthreads();
    }
    // Many tiles: whole ones, and the last one per SM cut in two, so that the SMs end together.  Few: cut so that each
    // SM gets about three units of few rows, one of more (a partial sum's way out and back costs rows; 48 rows of one
    // expert of 4096 x 4096: 24 us with three units to an SM, 18 with one).  A unit is long against that.
    const int head = total >= 3 * p.sms ? total - p.sms : 0;
    const int mrows = mt > 0 ? ceil_div(ceil_div(m, mt), 16) * 16 : 16;
    const int want = total >= 3 * p.sms ? 2 : mrows <= 32 ? ceil_div(3 * p.sms, max(total, 1)) : p.sms / max(total, 1);
    const int least = mrows <= 64 ? 8 : mrows <= 128 ? 16 : 32;
    int nu = max(1, min(want, p.kb / least));
    const int whole = min(max(head - (tile_end - tiles), 0), tiles);   // tiles of this expert that stay whole
    int ku = ceil_div(p.kb, nu);
    nu = ceil_div(p.kb, ku);
    const int blocks = nu > 1 ? (tiles - whole) * nu * (mrows / 16) : 0;
    const int part_end = block_scan<false>(min(blocks, p.part_cap + 1), warp_tot);
    if (nu > 1 && (blocks > p.part_cap || part_end > p.part_cap)) {    // no room for its partials: whole tiles
        nu = 1;
        ku = p.kb;
    }
    const int units = whole + (tiles - whole) * nu;
    const int unit_end = block_scan<false>(units, warp_tot);
    if (have) {
        ExpertRec r;
        r.lo = lo;
        r.m = m;
        r.tile0 = tile_end - tiles;
        r.unit0 = unit_end - units;
        r.part0 = part_end - blocks;
        r.nu = nu;
        r.ku = ku;
        r.mrows = mrows;
        p.rec[e] = r;
    }
    if (e == (int)blockDim.x - 1) {
        p.hdr[kHdrUnits] = unit_end;
        p.hdr[kHdrHead] = head;
        p.hdr[kHdrClaim] = 0;
        p.hdr[kHdrRowsLog] = rows_log;
    }
}

// ------------------------------------------------------------------ products

// A unit: K boxes k0 .. k1 - 1 of one tile.
struct Unit {
    int expert, n0;                 // weight rows n0 .. n0 + 127 of the expert
    int row0, rows;                 // rows of X in the tile
    int mrows;
    int k0, k1;
    int nu, part;                   // units of its tile, and the first one's partial block
    int split;                      // index of its tile among the split ones
    int j;                          // which of the tile's units
};

// (unit0 of the experts in shared memory: the last expert whose first unit is not past u has it -- experts
// without rows share their successor's unit0 and come before it)
__device__ __forceinline__ Unit unit_at(const ExpertParams &p, const int *unit0, int head, int rows_log, int u) {
    int lo = 0, hi = p.experts - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (unit0[mid] <= u) lo = mid;
        else hi = mid - 1;
    }
    const ExpertRec r = p.rec[lo];
    const int v = u - r.unit0;
    const int mt = m_tiles_of(r.m, rows_log);
    const int whole = min(max(head - r.tile0, 0), mt * p.n_g);
    Unit t;
    t.expert = lo;
    int tile;
    if (v < whole) {
        tile = v;
        t.nu = 1;
        t.j = 0;
        t.k0 = 0;
        t.k1 = p.kb;
        t.part = t.split = 0;
    } else {
        const int s = (v - whole) / r.nu;
        tile = whole + s;
        t.nu = r.nu;
        t.j = v - whole - s * r.nu;
        t.k0 = t.j * r.ku;
        t.k1 = min(p.kb, t.k0 + r.ku);
        t.part = r.part0 + s * r.nu * (r.mrows / 16);
        t.split = r.tile0 + tile - head;
    }
    // tiles of one weight column next to one another: they run at the same time and share it in L2
    const int g = tile / mt, i = tile - g * mt;
    t.n0 = g * kTileN;
    t.mrows = r.mrows;
    t.row0 = r.lo + i * r.mrows;
    t.rows = min(r.mrows, r.m - i * r.mrows);
    return t;
}

// True in one lane of the warp, which all lanes reach together.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0u;
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z,
                                            uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void tma_load_2d_at(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y,
                                               uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "l"(policy)
        : "memory");
}

// z / (1 + e^-z) * up by the hardware's exponential and division, relative error about 2^-20 up to |z| = 16, growing with
// the exponent's argument to 2^-17.5 at z = -87 (below that, where the value is under 2^-119, it is 0): the outputs are
// rounded to 2^-11 at the finest, and there are as many of these as outputs.
__device__ __forceinline__ float silu_mul(float z, float up) { return __fdividef(z, 1.f + __expf(-z)) * up; }

// Where outputs go: the launch's parameters, which the epilogue keeps in registers (read in its loop, they are
// fetched from constant memory again and again between the tcgen05 and barrier instructions, and miss).
template <typename T> struct Out {
    T *Y;
    long long stride;
    const float *row_scale;
    int N;
    bool silu;
};

// The scales of a chunk's rows, lane i that of row i (i + 16 too).
template <typename T> __device__ __forceinline__ float scales_of(const Out<T> &o, int row0, int cnt) {
    const int i = threadIdx.x & 15;
    return o.row_scale && i < cnt ? o.row_scale[row0 + i] : 1.f;
}

// Outputs of one thread: weight row n, rows row0 .. row0 + cnt - 1 of X (up to 16), sums v; scale from scales_of().
// A warp writes 64 bytes to a row (32 with SiLU*mul), and no branch is taken row by row: with one at every row a
// chunk of 16 rows took 2100 to 3700 clocks instead of 850.  With SiLU*mul lanes of gate rows finish rows 0 .. 7 and lanes of up
// rows 8 .. 15: each sends its partner (lane ^ 8) the eight sums that one needs.  Every lane of the warp calls this
// alike.
template <typename T>
__device__ __forceinline__ void emit_rows(const Out<T> &o, int n, int row0, int cnt, const float (&v)[16], float scale) {
    if (o.silu) {                                       // (N is a multiple of 16: a gate row in range has its up row)
        const bool up_lane = n & 8;
        const int first = up_lane ? 8 : 0;
        T *y = o.Y + (long long)(row0 + first) * o.stride + ((n >> 4) << 3) + (n & 7);
        const int mine = n < o.N ? cnt - first : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i, y += o.stride) {
            const float got = __shfl_xor_sync(0xffffffffu, up_lane ? v[i] : v[i + 8], 8);
            const float gate = up_lane ? got : v[i], up = up_lane ? v[i + 8] : got;
            const float s = __shfl_sync(0xffffffffu, scale, first + i);
            const T out = from_f32<T>(silu_mul(gate, up) * s);
            if (i < mine) *y = out;
        }
    } else {
        T *y = o.Y + (long long)row0 * o.stride + n;
        const int mine = n < o.N ? cnt : 0;
#pragma unroll
        for (int i = 0; i < 16; ++i, y += o.stride) {
            const T out = from_f32<T>(v[i] * __shfl_sync(0xffffffffu, scale, i));
            if (i < mine) *y = out;
        }
    }
}

__device__ __forceinline__ void ld_cg_rows4(const float *p, float *v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = ld_cg_f32(p + k * kTileN);
}

template <typename T>
__global__ void __launch_bounds__(kExThreads, 1) experts_kernel(const __grid_constant__ ExpertParams p) {
    extern __shared__ __align__(1024) uint8_t smem_dyn[];
    __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages], accf_bar[2], acce_bar[2], drain_bar;
    __shared__ Unit units[kUnitRing];                   // what the stages hold (expert -1: no more), by the producer
    __shared__ int acc_unit[2];                         // place there of an accumulator's (-1: no more), by the MMA thread
    __shared__ int unit0[kMaxExperts];
    __shared__ uint32_t tmem_base_sh;
    __shared__ volatile int abort_flag;
    __shared__ int last_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_dyn) + 1023) & ~uintptr_t(1023));
    int *const status = g_experts_status;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&accf_bar[b], 2);                 // tcgen05.commit and the MMA thread's unit number
            mbar_init(&acce_bar[b], kEpiSets * 4);
        }
        mbar_init(&drain_bar, 1);
        abort_flag = 0;
        fence_mbar_init();
        prefetch_tmap(&p.tmW);
    }
    if (warp == 1) tmem_alloc(&tmem_base_sh, kExTmemCols);
    pdl_wait();                                         // the plan is there, and whatever came before it
    for (int e = threadIdx.x; e < p.experts; e += kExThreads) unit0[e] = p.rec[e].unit0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = tmem_base_sh;
    const int n_units = p.hdr[kHdrUnits], head = p.hdr[kHdrHead], rows_log = p.hdr[kHdrRowsLog];
    const uint32_t ring_u = smem_u32(ring);

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (elect_one()) {
            const uint64_t pol_once = policy_evict_first(), pol_keep = policy_evict_normal();
            int s = 0, slot = 0;
            uint32_t ph = 0;
            long long issued = 0;
            bool aborted = false;
            if (p.stall_ns && blockIdx.x == 0) {
                // test hook: wait, bounded, on a word nothing sets, then abandon this CTA's work
                const unsigned long long t0 = globaltimer();
                while (ld_acquire_gpu(reinterpret_cast<const unsigned int *>(&status[kStatusStallFlag])) == 0u &&
                       globaltimer() - t0 <= p.stall_ns)
                    __nanosleep(256);
                record_error(status, kCodeTimeout, -1, kSiteStall);
                abort_flag = 1;
                aborted = true;
            }
            int u = (int)blockIdx.x;
            while (!aborted && u < n_units) {
                const Unit t = unit_at(p, unit0, head, rows_log, u);
                const int step = t.mrows <= kNarrow ? 2 : 1;
                // weights with one reader leave L2 first
                const uint64_t pol_w = p.rec[t.expert].m <= 1 << rows_log ? pol_once : pol_keep;
                // rows past the box in the MMA's N are what the stage held before, rows in it past the tile's another
                // expert's: nobody reads their sums
                const int box = box_of(t.rows);
                const CUtensorMap *const tmX = &p.tmX[box];
                const uint32_t box_bytes = (uint32_t)(kBoxW + box_rows(box) * kBK * 2);
                units[slot] = t;
                if (++slot == kUnitRing) slot = 0;
                int next = n_units;
                bool claimed = false;
                for (int k = t.k0; k < t.k1; k += step) {
                    if (!mbar_wait_bounded(&empty_bar[s], ph ^ 1, &abort_flag, kExWaitNs, status, t.expert, kSiteEmpty)) {
                        aborted = true;
                        break;
                    }
                    const int boxes = min(step, t.k1 - k);
                    mbar_arrive_expect_tx(&full_bar[s], boxes * box_bytes);
                    const uint32_t st = ring_u + (uint32_t)(s * kStageBytes);
                    for (int b = 0; b < boxes; ++b) {
                        tma_load_3d(st + b * kBoxW, &p.tmW, &full_bar[s], (k + b) * kBK, t.n0, t.expert, pol_w);
                        tma_load_2d_at(st + step * kBoxW + b * kNarrowX, tmX, &full_bar[s], (k + b) * kBK, t.row0, pol_keep);
                    }
                    ++issued;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                    if (!claimed && t.k1 - k <= kLead * step) {
                        next = (int)gridDim.x + (int)atom_add_relaxed_gpu(reinterpret_cast<unsigned int *>(&p.hdr[kHdrClaim]), 1u);
                        claimed = true;
                    }
                }
                u = next;
            }
            // every copy has landed before the CTA ends
            drain_issued(full_bar, kStages, issued, kExWaitNs, status);
            if (!aborted && mbar_wait_bounded(&empty_bar[s], ph ^ 1, &abort_flag, kExWaitNs, status, -1, kSiteEmpty)) {
                units[slot].expert = -1;
                mbar_arrive(&full_bar[s]);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        // One thread, and a stage's MMAs take as little as 128 clocks: nothing in the loop over a unit's stages but
        // the wait, the instructions and the commit. The thread is elected, not lane 0:
        // in a branch on the lane the compiler cannot tell that only one runs, and the thread spends 111 clocks on each
        // tcgen05.mma, 54 so.
        if (elect_one()) {
            int s = 0, slot = 0;
            uint32_t ph = 0, acc_i = 0;
            bool ok = true;
            const uint64_t desc0 = sw128_desc(ring_u);
            while (ok) {
                if (!mbar_wait_bounded(&full_bar[s], ph, &abort_flag, kExWaitNs, status, -1, kSiteFull)) break;
                const int here = slot, mrows = units[slot].mrows;
                const bool more = units[slot].expert >= 0;
                int left = units[slot].k1 - units[slot].k0;
                if (++slot == kUnitRing) slot = 0;
                const int buf = (int)(acc_i & 1u);
                if (!mbar_wait_bounded(&acce_bar[buf], ((acc_i >> 1) & 1u) ^ 1u, &abort_flag, kExWaitNs, status, -1, kSiteAcc)) break;
                if (!more) {
                    acc_unit[buf] = -1;
                    mbar_arrive(&accf_bar[buf]);
                    mbar_arrive(&accf_bar[buf]);
                    break;
                }
                const uint32_t idesc = p.idesc | ((uint32_t)(mrows >> 3) << 17);
                const uint32_t d = tmem_base + (uint32_t)(buf * kTileRows);
                const bool narrow = mrows <= kNarrow;
                const uint64_t x_off = (uint64_t)(((narrow ? 2 : 1) * kBoxW) >> 4);
                uint32_t add = 0u;
                tc_fence_after();
                for (;;) {
                    const uint64_t a = desc0 + (uint64_t)(s * (kStageBytes >> 4)), b = a + x_off;
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k) {        // 16 K elements are 32 bytes of a swizzle row
                        tc_mma(d, a + 2u * k, b + 2u * k, idesc, add);
                        add = 1u;
                    }
                    if (narrow && left > 1) {
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k)
                            tc_mma(d, a + (kBoxW >> 4) + 2u * k, b + (kNarrowX >> 4) + 2u * k, idesc, 1u);
                    }
                    tc_commit(&empty_bar[s]);
                    left -= narrow ? 2 : 1;
                    if (++s == kStages) {
                        s = 0;
                        ph ^= 1;
                    }
                    if (left <= 0) break;
                    if (!mbar_wait_bounded(&full_bar[s], ph, &abort_flag, kExWaitNs, status, -1, kSiteFull)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                }
                if (!ok) break;
                acc_unit[buf] = here;
                mbar_arrive(&accf_bar[buf]);
                tc_commit(&accf_bar[buf]);
                ++acc_i;
            }
            // all MMAs are complete before tensor memory is released
            tc_commit(&drain_bar);
            volatile int never = 0;
            mbar_wait_bounded(&drain_bar, 0, &never, kExWaitNs, status, -1, kSiteDrain);
        }
    } else {
        // ------------------------------------------------------------ epilogue
        // Two sets of four warps, each with every other 16 rows of a tile.
        const int set = (warp - 2) >> 2;
        const int q = warp & 3;                         // TMEM lane quadrant this warp may read
        const int row = q * 32 + lane;                  // weight row within the tile
        const bool leader = threadIdx.x == 64;
        constexpr int kStep = kEpiSets * 16;
        const Out<T> out = {static_cast<T *>(p.Y), p.y_stride, p.row_scale, p.N, p.silu != 0};
        float *const parts = p.part;
        for (uint32_t i = 0;; ++i) {
            const int buf = (int)(i & 1u);
            const bool ab = !mbar_wait_bounded(&accf_bar[buf], (i >> 1) & 1u, &abort_flag, kExWaitNs, status, -1, kSiteAcc);
            const int u = ab ? -1 : acc_unit[buf];
            if (vote_or(u < 0, 1, kEpiSets * 128)) break;   // the eight warps stop together
            tc_fence_after();
            const Unit t = units[u];
            const uint32_t taddr = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf * kTileRows);
            float *part = parts + ((size_t)t.part + (size_t)t.j * (t.mrows / 16)) * (16 * kTileN) + row;
            uint32_t r[16], ahead[16];
            if (set * 16 < t.rows) tmem_ld16(taddr + (uint32_t)(set * 16), ahead);
#pragma unroll 1
            for (int c = set * 16; c < t.rows; c += kStep) {
                const int cnt = min(16, t.rows - c);
                const float scale = t.nu == 1 ? scales_of(out, t.row0 + c, cnt) : 1.f;
                tmem_ld_wait16(ahead);
#pragma unroll
                for (int k = 0; k < 16; ++k) r[k] = ahead[k];
                if (c + kStep < t.rows) tmem_ld16(taddr + (uint32_t)(c + kStep), ahead);    // under this chunk's work
                float v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[k]);
                if (t.nu == 1) {
                    emit_rows(out, t.n0 + row, t.row0 + c, cnt, v, scale);
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        if (k < cnt) part[(size_t)(c + k) * kTileN] = v[k];
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acce_bar[buf]);
            if (t.nu == 1) continue;
            // the tile's last unit to arrive adds all partials, in K order
            named_bar_sync(2, kEpiSets * 128);
            if (leader) last_flag = atom_add_acqrel_gpu(&p.tile_cnt[t.split], 1u) == (unsigned int)(t.nu - 1) ? 1 : 0;
            named_bar_sync(2, kEpiSets * 128);
            if (!last_flag) continue;
            const float *from = parts + (size_t)t.part * (16 * kTileN) + row;
            const size_t step = (size_t)(t.mrows / 16) * (16 * kTileN);
#pragma unroll 1
            for (int c = set * 16; c < t.rows; c += kStep) {
                const int cnt = min(16, t.rows - c);
                const float scale = scales_of(out, t.row0 + c, cnt);
                float v[16];
                const float *f = from + (size_t)c * kTileN;
                for (int j = 0; j < t.nu; j += 2, f += 2 * step) {
                    // rows by fours, those past the tile's whatever the block of 16 holds: nobody reads their sums
                    float w[2][16];
                    const bool two = j + 1 < t.nu;
#pragma unroll
                    for (int k = 0; k < 16; k += 4)
                        if (k < cnt) {
                            ld_cg_rows4(f + k * kTileN, w[0] + k);
                            if (two) ld_cg_rows4(f + step + k * kTileN, w[1] + k);
                        }
#pragma unroll
                    for (int k = 0; k < 16; ++k) v[k] = j == 0 ? w[0][k] : v[k] + w[0][k];
                    if (two)
#pragma unroll
                        for (int k = 0; k < 16; ++k) v[k] += w[1][k];
                }
                emit_rows(out, t.n0 + row, t.row0 + c, cnt, v, scale);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // Only now, when this CTA is through with the scratch (its partials were performed before their unit's arrival was
    // counted): the next call may be one that waits for nothing (WSM_FLAG_INDEPENDENT), and its outputs may lie in
    // the scratch, which is the caller's again once this call has returned.
    pdl_launch_dependents();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem_base, kExTmemCols);
}

// ------------------------------------------------------------------ host side

struct ExLayout {
    size_t rec, cnt, part, total;
    int cnt_cap, part_cap;
};
ExLayout experts_layout(int rows, int experts, int sms) {
    ExLayout l;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const int mrows = (std::min(rows, kTileRows) + 15) / 16 * 16;
    l.cnt_cap = 3 * sms;                                // split tiles: fewer than three per SM
    // units of split tiles: under six per SM; at most 32 MB of partials (tiles that find no room stay whole)
    l.part_cap = std::min(6 * sms * (mrows / 16), 4096);
    l.rec = kHdrBytes;
    l.cnt = up(l.rec + sizeof(ExpertRec) * (size_t)experts);
    l.part = up(l.cnt + 4 * (size_t)l.cnt_cap);
    l.total = l.part + (size_t)l.part_cap * (16 * kTileN * 4);
    return l;
}

}  // namespace

wsm_status experts_status_ptr(void **p) {
    WSM_OP_CUDA(cudaGetSymbolAddress(p, g_experts_status));
    return WSM_OK;
}

wsm_status experts_error_ptr(void **p) {
    WSM_OP_CUDA(cudaGetSymbolAddress(p, g_experts_error));
    return WSM_OK;
}

}  // namespace wsm

using namespace wsm;

extern "C" {

size_t wsm_expert_gemm_workspace_bytes(int rows, int experts) {
    if (rows < 0 || experts < 1 || experts > kMaxExperts) {
        op_fail(WSM_ERR_UNSUPPORTED, "expert products take up to %d experts and no negative rows (got %d, %d)", kMaxExperts, experts, rows);
        return 0;
    }
    int dev, sms;
    if (device_sms(&dev, &sms) != WSM_OK) return 0;
    return experts_layout(rows, experts, sms).total;
}

wsm_status wsm_expert_gemm(const wsm_experts *a, wsm_stream_t stream_) {
    if (!a) return op_fail(WSM_ERR_INVALID, "the arguments must be non-null");
    if (a->rows < 0 || a->experts < 1 || a->N < 1)
        return op_fail(WSM_ERR_INVALID, "rows %d, experts %d, N %d: no negative rows, and an expert and an output at least", a->rows, a->experts, a->N);
    if (a->experts > kMaxExperts) return op_fail(WSM_ERR_UNSUPPORTED, "%d experts: up to %d are", a->experts, kMaxExperts);
    if (a->K < 8 || a->K % 8) return op_fail(WSM_ERR_UNSUPPORTED, "unsupported K=%d (need K>=8, K%%8==0)", a->K);
    if (a->dtype != WSM_DTYPE_BF16 && a->dtype != WSM_DTYPE_FP16)
        return op_fail(WSM_ERR_UNSUPPORTED, "element type %d: bf16 and fp16 are", a->dtype);
    if (a->epilogue != WSM_EPI_NONE && a->epilogue != WSM_EPI_SILU_MUL)
        return op_fail(WSM_ERR_UNSUPPORTED, "epilogue %d: WSM_EPI_NONE and WSM_EPI_SILU_MUL are", a->epilogue);
    if (a->epilogue == WSM_EPI_SILU_MUL && a->N % 16)
        return op_fail(WSM_ERR_UNSUPPORTED, "SiLU*mul needs N a multiple of 16 (got %d)", a->N);
    if (a->rows == 0) return WSM_OK;
    if (!a->X || !a->W || !a->Y || !a->offsets || !a->workspace)
        return op_fail(WSM_ERR_INVALID, "X, W, Y, offsets and workspace must be non-null device pointers");
    if (!aligned_to(a->X, 16) || !aligned_to(a->W, 16) || !aligned_to(a->workspace, 16))
        return op_fail(WSM_ERR_ALIGN, "X, W and workspace must be 16-byte aligned");
    if (!aligned_to(a->Y, 2) || !aligned_to(a->offsets, 4) || !aligned_to(a->row_scale, 4))
        return op_fail(WSM_ERR_ALIGN, "Y, offsets and row_scale must be aligned to their elements");
    // a stride that no second row, output or expert uses may be anything
    const long long K = a->K, xs = a->rows > 1 ? a->x_stride : K, wr = a->N > 1 ? a->w_strides[1] : K,
                    we = a->experts > 1 ? a->w_strides[0] : (long long)a->N * std::max(wr, K);
    const int y_cols = a->epilogue == WSM_EPI_SILU_MUL ? a->N / 2 : a->N;
    if (xs % 8 || wr % 8 || we % 8) return op_fail(WSM_ERR_ALIGN, "the strides of X and W must be multiples of 16 bytes");
    if (xs < K || wr < K || we < (long long)(a->N - 1) * wr + K || (a->rows > 1 && a->y_stride < y_cols))
        return op_fail(WSM_ERR_INVALID, "rows of X, W or Y overlap: strides %lld, %lld, %lld, %lld", xs, wr, we, a->y_stride);
    if (xs >= (1ll << 39) || wr >= (1ll << 39) || we >= (1ll << 39)) return op_fail(WSM_ERR_UNSUPPORTED, "a stride is too large");
    // tiles and their units are counted in 32 bits
    const long long n_g = ((long long)a->N + kTileN - 1) / kTileN;
    if (a->rows > (1 << 30) || K > (1 << 30) || n_g * (a->rows / kTileRows + a->experts + 1) >= (1ll << 30))
        return op_fail(WSM_ERR_UNSUPPORTED, "%d rows by %d outputs of %d terms are too many", a->rows, a->N, a->K);
    int dev, sms;
    wsm_status st = device_sms(&dev, &sms);
    if (st != WSM_OK) return st;
    const ExLayout l = experts_layout(a->rows, a->experts, sms);
    if (a->workspace_bytes < l.total)
        return op_fail(WSM_ERR_NOMEM, "workspace of %zu bytes is smaller than the %zu needed", a->workspace_bytes, l.total);

    const bool bf = a->dtype == WSM_DTYPE_BF16;
    const CUtensorMapDataType type = bf ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
    ExpertParams p = {};
    {
        const cuuint64_t dims[3] = {(cuuint64_t)K, (cuuint64_t)a->N, (cuuint64_t)a->experts};
        const cuuint64_t strides[2] = {(cuuint64_t)wr * 2, (cuuint64_t)we * 2};
        const cuuint32_t box[3] = {kBK, kTileN, 1};
        if ((st = encode_tiled(&p.tmW, type, 3, a->W, dims, strides, box)) != WSM_OK) return st;
    }
    for (int i = 0; i <= box_of(std::min(a->rows, kTileRows)); ++i) {   // no tile is higher
        const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)a->rows};
        const cuuint64_t strides[1] = {(cuuint64_t)xs * 2};
        const cuuint32_t box[2] = {kBK, (cuuint32_t)box_rows(i)};
        if ((st = encode_tiled(&p.tmX[i], type, 2, a->X, dims, strides, box)) != WSM_OK) return st;
    }
    uint8_t *ws = static_cast<uint8_t *>(a->workspace);
    p.Y = a->Y;
    p.offsets = a->offsets;
    p.row_scale = a->row_scale;
    p.y_stride = a->y_stride;
    p.hdr = reinterpret_cast<int *>(ws);
    p.rec = reinterpret_cast<ExpertRec *>(ws + l.rec);
    p.tile_cnt = reinterpret_cast<unsigned int *>(ws + l.cnt);
    p.part = reinterpret_cast<float *>(ws + l.part);
    p.part_cap = l.part_cap;
    p.cnt_cap = l.cnt_cap;
    p.rows = a->rows;
    p.experts = a->experts;
    p.N = a->N;
    p.K = a->K;
    p.kb = (a->K + kBK - 1) / kBK;
    p.n_g = (int)n_g;
    p.silu = a->epilogue == WSM_EPI_SILU_MUL;
    p.sms = sms;
    // fp32 accumulators, A and B of one 16-bit type, both K-major, M = 128
    p.idesc = (1u << 4) | (bf ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)(kTileN >> 4) << 24);
    p.stall_ns = take_launch_stall();
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
    const int plan_threads = (a->experts + 31) / 32 * 32;
    if ((st = op_launch(&experts_plan_kernel, dim3(1), plan_threads, 0, stream, p)) != WSM_OK) return st;
    constexpr int kSmem = kStages * kStageBytes + 1024;
    static volatile bool done[2][kMaxOpDevices] = {};
    if (bf) {
        if ((st = op_allow_smem(&experts_kernel<__nv_bfloat16>, kSmem, dev, done[0])) != WSM_OK) return st;
        return op_launch(&experts_kernel<__nv_bfloat16>, dim3((unsigned)sms), kExThreads, kSmem, stream, p);
    }
    if ((st = op_allow_smem(&experts_kernel<__half>, kSmem, dev, done[1])) != WSM_OK) return st;
    return op_launch(&experts_kernel<__half>, dim3((unsigned)sms), kExThreads, kSmem, stream, p);
}

}  // extern "C"
