// The whole layer for a few tokens (T <= 16) in one persistent kernel.
//
// Decoding a few tokens is bound by the bytes of the experts they reach, so
// the kernel is a stream of weight rows through every SM that nothing
// interrupts: a warp loads pieces of 128 weight rows x 128 bytes by TMA into a
// ring in shared memory, and tcgen05 multiplies them in place, the weights as
// the 128-row operand and the tokens as a narrow one.  No thread touches a
// weight; what the other warps do per piece is a few copies of the token side.
// One block per SM, launched cooperatively; the phases are separated by grid
// barriers, and since weights do not depend on what the barriers wait for, the
// ring keeps filling across them:
//   1  router logits: (expert, slice of d) dot products in fp32, partial sums
//      per slice; x into the operand form of the weights' type;
//   -- barrier; every block then selects the top-K of all tokens for itself
//      (slices added in order) and builds the list of experts reached;
//   2  h = SiLU(W1 x + b1), written per (token, slot);
//   -- barrier; FP8 and MXFP4: h into the operand form, barrier;
//   3  out = sum over the experts of gate * (W2 h + b2), shared experts
//      included.
// Phases 2 and 3 are one sequence each of tiles of 128 result rows (phase 2:
// of every expert's W1; phase 3: of the output, through every expert's W2),
// each a run of slots (two pieces of K).  Every block takes the same number of
// slots; a tile that crosses a block boundary is summed from its blocks' parts,
// in block order, by whichever of them finishes last.
//
// Operand forms (products exact, sums in fp32):
//   bf16   weights, x and h in bf16 (kind::f16);
//   FP8    e4m3 (kind::mxf8f6f4.block_scale); x and h quantised to e4m3 per 128
//          columns; all scales are powers of two and go to the tensor core;
//   MXFP4  packed E2M1 with its E8M0 scales (kind::mxf4.block_scale).  x and h
//          are not quantised: per 32 columns they are split into five E2M1
//          planes, each the nearest E2M1 value of what the planes before it
//          left, at scales s, s/4, s/32, s/256, s/2048.  A plane's remainder is
//          at most half of the step at its largest magnitude (1, then 1/2 of
//          the next plane's unit), so the five stand for the value to within
//          s / 4096 <= amax / 12288.  A token is then five columns, which the
//          tensor core has to spare.
//
// Per block (320 threads):
//   warps 0..3  epilogue (thread = row);   warps 4..7  token side: operand
//   rows and all scales by cp.async;       (both: phase 1, the selection and
//   the conversion of h)   warp 8  weights by TMA;   warp 9  MMA issue.
// The weights stream past L2, so at every call the code itself comes from HBM:
// a phase's first instructions cost as much as its first weights.  The role
// loops therefore run both phases through the same code (measured: 172 KB of
// code took 10 us to select the experts of one token and 7 us from there to
// the first weights).
// Every wait is bounded (common.cuh); after a wait gives up, the warps skip
// the remaining work but keep meeting at the block's barriers.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cstring>
#include "internal.h"
#include "mxfp4.cuh"

namespace moe {
namespace {

constexpr int CW = 8;                          // general warps
constexpr int CT = CW * 32;
constexpr int W_TMA = 8, W_MMA = 9;
constexpr int THREADS = CT + 64;
constexpr int EPI = 128;                       // epilogue threads, and token-side threads
constexpr int NP = 2;                          // pieces per slot
constexpr int MAX_SLOTS = 5, PIECE_BYTES = 16384;
constexpr int MAX_T = MOE_FEW_MAX_TOKENS;
constexpr int MAX_BLOCKS = 256;
constexpr int PLANES = 5;                      // MXFP4: columns per token
constexpr uint32_t ACC_COLS = 96, SF_COL0 = 2 * ACC_COLS, SF_COLS = 32, TMEM_COLS = 256;
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;

constexpr int OFF_IDX = 0;                                     // [16][16] int
constexpr int OFF_GATE = OFF_IDX + MAX_T * 16 * 4;             // [16][16] float
constexpr int OFF_MASK = OFF_GATE + MAX_T * 16 * 4;            // [256] tokens kept, per expert
constexpr int OFF_KPACK = OFF_MASK + 256 * 4;                  // [256] 4 bits per token: its slot
constexpr int OFF_ACT = OFF_KPACK + 256 * 8;                   // [256] experts reached, ascending
constexpr int OFF_COUNT = OFF_ACT + 256 * 4;                   // [256] slots that name the expert
constexpr int OFF_OUT = OFF_COUNT + 256 * 4;                   // [16][128] fp32 sums of a tile
constexpr int OFF_BAR = OFF_OUT + MAX_T * 128 * 4;             // full, empty [MAX_SLOTS]; accf, acce [2]; drain
constexpr int OFF_MISC = OFF_BAR + (2 * MAX_SLOTS + 5) * 8;    // abort flag, n_active, tmem address, last flag, 8 warp counts
constexpr int OFF_RING = (OFF_MISC + 64 + 1023) & ~1023;
constexpr int RING_BYTES = 206 * 1024;
constexpr int SMEM_ALLOC = OFF_RING + RING_BYTES + 1024;
static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory budget");
static_assert(OFF_KPACK % 8 == 0 && OFF_BAR % 8 == 0, "alignment");
static_assert(SF_COL0 + 2 * SF_COLS <= TMEM_COLS && PLANES * MAX_T + 3 <= ACC_COLS, "tensor memory budget");

// grid-wide counters in the workspace, zero between launches
enum { CTR_BAR = 0, CTR_EXIT = 3, CTR_ABORT = 4, CTR_WORDS = 5, CTR_TILE = 64 };

struct __align__(64) FewParams {
    CUtensorMap w1, w2, ws1, ws2;
    const __nv_bfloat16* x;
    const float* W_r;
    const float* logit_bias;      // added to the logits, or nullptr
    const float* sel_bias;        // added to the selection keys, or nullptr
    const void *w1s, *w2s, *ws1s, *ws2s;
    const float *b1, *b2, *bs1, *bs2;
    __nv_bfloat16* out;
    float *f, *P, *loss;
    int32_t *topk_idx, *counts;   // or nullptr
    float* gates;                 // or nullptr
    // workspace
    int32_t* status;
    uint32_t* ctr;
    float* part;                  // (ks, T, E) partial logits
    float* prob;                  // (T, 256) softmax of the logits
    uint8_t* xq;                  // x in operand form (bf16: x itself)
    uint8_t* xs;                  // its scales: FP8 a word per 128 columns, MXFP4 a byte per 32
    float* h32;                   // fp32 h: (T K, dff), then (S T, dffs)
    uint8_t* hq;                  // h in operand form, same rows (bf16: the only form)
    uint8_t* hs;                  // its scales
    float* sums;                  // (blocks, 2, T, 128) parts of tiles that cross blocks
    float alpha;
    int T, d, E, K, dff, S, dffs, capacity, slot_major, passthrough;
    int ks, slice;                // router slices of d and their length
    int slots, slot_bytes;        // ring
};

enum { M_BF16 = 0, M_FP8 = 1, M_FP4 = 2 };

// KP: elements of K in a piece (128 bytes of a weight row); P: columns per
// token; SF: bytes of scales per piece (weights', then tokens')
template <int MODE> struct Form;
template <> struct Form<M_BF16> { static constexpr int KP = 64, P = 1, SF = 0; };
template <> struct Form<M_FP8> { static constexpr int KP = 128, P = 1, SF = 1024; };
template <> struct Form<M_FP4> { static constexpr int KP = 256, P = PLANES, SF = 2048; };

__host__ __device__ constexpr int round16(int v) { return (v + 15) & ~15; }

__device__ __forceinline__ void bar_general() { asm volatile("bar.sync 1, %0;" :: "n"(CT) : "memory"); }

__device__ __forceinline__ void bar_tokens() { asm volatile("bar.sync 3, %0;" :: "n"(EPI) : "memory"); }
__device__ __forceinline__ void bar_epilogue() { asm volatile("bar.sync 2, %0;" :: "n"(EPI) : "memory"); }

__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" :: "r"(smem_u32(dst)), "l"(src) : "memory");
}

__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(dst)), "l"(src) : "memory");
}

// Arrives on bar once this thread's earlier cp.async copies have landed (the
// barrier's count includes the arrival).
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// ---------------------------------------------------------------- operand form of x and h

// 128 consecutive values of row `row` (a token of x, a slot of h) starting at
// column col, four per lane, into the operand form of rows of k columns.
template <int MODE>
__device__ __noinline__ void store_block(float4 v4, uint8_t* q, uint8_t* scales, size_t row, int k, int col, int lane) {
    float v[4] = {v4.x, v4.y, v4.z, v4.w};
    if (MODE == M_FP8) {
        // as the dispatch quantiser: fmaxf does not count a NaN
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) a = fmaxf(a, fabsf(v[j]));
        const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(a));
        const float sc = pow2_scale_448(__uint_as_float(m)), inv = inv_pow2(sc);
        const uint32_t lo = f32x2_to_e4m3x2(v[0] * inv, v[1] * inv), hi = f32x2_to_e4m3x2(v[2] * inv, v[3] * inv);
        reinterpret_cast<uint32_t*>(q + row * k + col)[lane] = lo | (hi << 16);
        // the scale's UE8M0 byte, once per 32 columns
        if (lane == 0) reinterpret_cast<uint32_t*>(scales)[row * (k / 128) + col / 128] =
            (__float_as_uint(sc) >> 23) * 0x01010101u;
    } else {
        // eight lanes have a block of 32
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const uint32_t b = mxfp4_scale_byte(m);
        const float inv = mxfp4_inv_scale(b == 255u ? 127u : b);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] *= inv;
#pragma unroll 1
        for (int pl = 0; pl < PLANES; ++pl) {
            // scale exponents b, b - 2, b - 5, b - 8, b - 11; a plane below the
            // smallest scale holds nothing
            const int e = static_cast<int>(b) - (pl == 0 ? 0 : 3 * pl - 1);
            const uint32_t codes = b == 255u || e < 0 ? 0u : f32x4_to_e2m1x4(v[0], v[1], v[2], v[3]);
            float back[4];
            e2m1x4_to_f32(codes, back);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = (v[j] - back[j]) * (pl == 0 ? 4.f : 8.f);
            const size_t r = row * PLANES + pl;
            reinterpret_cast<uint16_t*>(q + (r * k + col) / 2)[lane] = static_cast<uint16_t>(codes);
            if ((lane & 7) == 0)
                scales[(r * k + col) / 32 + lane / 8] = static_cast<uint8_t>(b == 255u ? 255 : max(e, 0));
        }
    }
}

// ---------------------------------------------------------------- grid barrier

struct Ctx {
    const FewParams& p;
    uint8_t* smem;
    uint64_t* full;
    uint64_t* empty;
    volatile int* abort_flag;
    int tid, warp, lane;
};

// Bounded wait on a phase of one of the block's barriers.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, const Ctx& c) {
    return mbar_wait_bounded(bar, parity, c.abort_flag, c.p.status, kWaitNs);
}

// The general warps of all blocks.  Writes before it are visible to reads
// (through L2) after it.
__device__ __noinline__ void grid_barrier(uint32_t* ctrs, int which, int32_t* status, volatile int* abort_flag, int tid) {
    bar_general();
    if (tid == 0) {
        uint32_t* ctr = ctrs + CTR_BAR + which;
        __threadfence();
        atomicAdd(ctr, 1u);
        if (*abort_flag) atomicExch(ctrs + CTR_ABORT, 1u);
        uint64_t t0 = 0;
        for (uint32_t it = 1; !*abort_flag && ld_acquire(ctr) < gridDim.x; ++it) {
            if ((it & 255u) == 0) {
                const uint64_t now = global_timer_ns();
                if (t0 == 0) t0 = now;
                if (ld_acquire(ctrs + CTR_ABORT)) *abort_flag = 1;
                else if (now - t0 > kWaitNs) {
                    *abort_flag = 1;
                    set_device_status(status, MOE_DEV_TIMEOUT);
                    atomicExch(ctrs + CTR_ABORT, 1u);
                }
            }
        }
        __threadfence();
    }
    bar_general();
}

// ---------------------------------------------------------------- jobs

// A job: a run of slots of one tile and one matrix: pieces p0 .. p1 - 1 of K
// (128 bytes of every row each) of rows row0 .. row0 + 127, for the tokens of
// `mask`; the j-th of them has the columns j P .. j P + P - 1.
struct Job {
    int shared;           // 1: shared expert
    int mat, row0;
    int n, k;             // the matrix: n rows of k columns
    int p0, p1;
    uint32_t mask;
    uint64_t kpack;       // routed: the tokens' slots
    bool ends;            // the block's last job of this tile
    // the blocks that have slots of this tile
    int block0, block1;
};

// Row of h for token t of a job.
__device__ __forceinline__ int h_row(const Ctx& c, const Job& j, int t) {
    return j.shared ? j.mat * c.p.T + t : t * c.p.K + (static_cast<int>(j.kpack >> (4 * t)) & 15);
}

// This block's share of a phase's slots, job by job.  Phase 2: matrix by
// matrix, its tiles, their slots of K = d.  Phase 3: tile by tile, the shared
// experts' slots, then those of the experts reached.
template <int MODE>
struct Jobs {
    const Ctx& c;
    const bool third;     // phase 3
    int at, end;
    int each, extra;      // slots of a block; the first `extra` blocks have one more
    int ss, sr;           // slots of a shared, a routed matrix per tile
    int ts, tr;           // phase 2: tiles of a shared, a routed matrix
    int tile;             // phase 3: slots of a tile
    static __device__ __forceinline__ int slots_of(int k) { return (k + NP * Form<MODE>::KP - 1) / (NP * Form<MODE>::KP); }
    __device__ __forceinline__ Jobs(const Ctx& c_, int phase, int n_active) : c(c_), third(phase == 3) {
        const FewParams& p = c.p;
        int all;
        if (!third) {
            ss = sr = slots_of(p.d);
            ts = (p.dffs + 127) / 128;
            tr = (p.dff + 127) / 128;
            tile = 1;
            all = (p.S * ts + n_active * tr) * sr;
        } else {
            ss = slots_of(p.dffs);
            sr = slots_of(p.dff);
            ts = tr = 1;
            tile = p.S * ss + n_active * sr;
            all = (p.d + 127) / 128 * tile;
        }
        // with fewer slots than blocks the last blocks have none, so that every
        // block between a tile's first and last has some of it
        const int b = blockIdx.x;
        each = all / static_cast<int>(gridDim.x);
        extra = all - each * static_cast<int>(gridDim.x);
        at = b * each + min(b, extra);
        end = at + each + (b < extra ? 1 : 0);
    }
    // the block that has slot u
    __device__ __forceinline__ int block_of(int u) const {
        const int v = u - extra * (each + 1);
        return v < 0 ? u / (each + 1) : extra + v / each;
    }
    __device__ __forceinline__ bool next(Job& j) {
        if (at >= end) return false;
        const FewParams& p = c.p;
        int u = at, first = 0;
        if (third) {
            j.row0 = u / tile * 128;
            first = u / tile * tile;
            u -= first;
        }
        const int n_shared = p.S * ts * ss;
        j.shared = u < n_shared;
        if (!j.shared) u -= n_shared;
        const int per = j.shared ? ss : sr, tiles = j.shared ? ts : tr;
        const int run = u / per, s0 = u - run * per;           // (matrix, tile), first slot of it
        const int m = run / tiles;
        if (!third) {
            j.row0 = (run - m * tiles) * 128;
            first = at - s0;
        }
        const int take = min(per - s0, end - at);
        j.mat = j.shared ? m : reinterpret_cast<const int*>(c.smem + OFF_ACT)[m];
        j.mask = j.shared ? (1u << p.T) - 1u : reinterpret_cast<const uint32_t*>(c.smem + OFF_MASK)[j.mat];
        j.kpack = j.shared ? 0 : reinterpret_cast<const uint64_t*>(c.smem + OFF_KPACK)[j.mat];
        const int inner = j.shared ? p.dffs : p.dff;
        j.n = third ? p.d : inner;
        j.k = third ? inner : p.d;
        j.p0 = s0 * NP;
        j.p1 = min((s0 + take) * NP, (j.k + Form<MODE>::KP - 1) / Form<MODE>::KP);
        at += take;
        const int last = first + (third ? tile : per) - 1;
        j.ends = at == end || at > last;
        j.block0 = block_of(first);
        j.block1 = block_of(last);
        return true;
    }
};

struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int slots) { if (++slot == slots) { slot = 0; phase ^= 1u; } }
};

// A slot of the ring: NP pieces of weights, the tokens' rows of each, the
// scales of each.
__device__ __forceinline__ uint8_t* slot_at(const Ctx& c, int slot) { return c.smem + OFF_RING + slot * c.p.slot_bytes; }
template <int MODE>
__device__ __forceinline__ int rows_bytes(const Ctx& c) { return round16(c.p.T * Form<MODE>::P) * 128; }
template <int MODE>
__device__ __forceinline__ int scales_at(const Ctx& c) { return NP * (PIECE_BYTES + rows_bytes<MODE>(c)); }

// ---------------------------------------------------------------- weights (one warp)

// Loads a job's weights; false after a wait gave up.
template <int MODE>
__device__ __forceinline__ bool load_weights(const Ctx& c, const Job& j, const CUtensorMap* map, Ring& ring) {
    constexpr int ELEMS = MODE == M_BF16 ? 64 : 128;        // map elements (bf16, or bytes) per piece
    for (int s = j.p0; s < j.p1; s += NP) {
        uint64_t* full = c.full + ring.slot;
        const int np = min(NP, j.p1 - s);
        int ok = 1;
        if (c.lane == 0) {
            ok = wait(c.empty + ring.slot, ring.phase ^ 1u, c);
            if (ok) mbar_arrive_expect_tx(full, static_cast<uint32_t>(np * PIECE_BYTES));
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
        if (c.lane < np)
            tma_load_3d(slot_at(c, ring.slot) + c.lane * PIECE_BYTES, map, full, (s + c.lane) * ELEMS, j.row0, j.mat);
        ring.next(c.p.slots);
    }
    return true;
}

// ---------------------------------------------------------------- token side (128 threads)

// The tokens' operand rows and the scales of every piece of a phase's jobs,
// copied by cp.async; the copies' own completion arrives on the slot's barrier.
// (The tensor core reads them through the async proxy: the MMA thread, which
// has nothing else in flight, makes the proxy fence.  Made here it would wait
// for the copies just issued: measured 1000 cycles a piece.)
template <int MODE>
__device__ __forceinline__ void load_tokens(const Ctx& c, int phase, int n_active, size_t h_shared, Ring& ring, bool& ok) {
    constexpr int P = Form<MODE>::P, KP = Form<MODE>::KP;
    const FewParams& p = c.p;
    const bool third = phase == 3;
    const int i = c.tid - EPI;
    const int q = i & 7;                                       // 16-byte chunk of a row's 128 bytes
    const int word = 16 * (i & 31) + 4 * (i >> 5);             // row i's word in 512 bytes of scales
    const int row_bytes = rows_bytes<MODE>(c), sf_at = scales_at<MODE>(c);
    Jobs<MODE> jobs(c, phase, n_active);
    Job j;
    while (ok && jobs.next(j)) {
        const int rows = __popc(j.mask) * P;
        // bytes of an operand row of j.k columns
        const size_t pitch = MODE == M_BF16 ? 2 * static_cast<size_t>(j.k) : MODE == M_FP8 ? j.k : j.k / 2;
        const int kq = MODE == M_FP8 ? j.k / 128 * 4 : j.k / 32;   // and of its scales
        // shared experts' rows of h follow the routed ones, at their own width
        const uint8_t* data = third ? p.hq : p.xq;
        const uint8_t* sc = third ? p.hs : p.xs;
        if (third && j.shared) {
            const size_t skip = h_shared * P;
            data += MODE == M_BF16 ? 2 * skip : MODE == M_FP8 ? skip : skip / 2;
            sc += MODE == M_FP8 ? skip / 128 * 4 : skip / 32;
        }
        auto operand_row = [&](int n) {                        // of column n
            uint32_t m = j.mask;
            for (int z = n / P; z > 0; --z) m &= m - 1;
            const int t = __ffs(m) - 1;
            return static_cast<size_t>((third ? h_row(c, j, t) : t) * P + n % P);
        };
        const uint8_t* src[P];                                 // 16 rows at a time, 16 P in all
#pragma unroll
        for (int b = 0; b < P; ++b) {
            const int n = (i >> 3) + 16 * b;
            src[b] = n < rows ? data + operand_row(n) * pitch + 16 * q : nullptr;
        }
        const uint8_t* bs = nullptr;                           // scales of column i
        const uint8_t* as = nullptr;                           // scales of weight row i
        if (MODE != M_BF16) {
            if (i < rows) bs = sc + operand_row(i) * kq;
            if (j.row0 + i < j.n) {
                const uint8_t* w = static_cast<const uint8_t*>(third ? (j.shared ? p.ws2s : p.w2s) : (j.shared ? p.ws1s : p.w1s));
                as = MODE == M_FP8 ? w + (static_cast<size_t>(j.mat) * (j.n / 128) + j.row0 / 128) * kq
                                   : w + (static_cast<size_t>(j.mat) * j.n + j.row0 + i) * kq;
            }
        }
        float wsc[NP];                                         // FP8: the tile's weight scales, a slot ahead
        auto fetch = [&](int s) {
#pragma unroll
            for (int r = 0; r < NP; ++r)
                wsc[r] = s + r < j.p1 ? __ldg(reinterpret_cast<const float*>(as) + s + r) : 0.f;
        };
        if (MODE == M_FP8) fetch(j.p0);
        for (int s = j.p0; s < j.p1; s += NP) {
            int w = 1;
            if (c.lane == 0) w = wait(c.empty + ring.slot, ring.phase ^ 1u, c);
            if (!__shfl_sync(0xffffffffu, w, 0)) { ok = false; break; }
            uint8_t* slot = slot_at(c, ring.slot);
#pragma unroll
            for (int r = 0; r < NP; ++r) {
                const int piece = s + r;
                if (piece >= j.p1) break;
                uint8_t* bdst = slot + NP * PIECE_BYTES + r * row_bytes;
#pragma unroll
                for (int b = 0; b < P; ++b) {
                    const int n = (i >> 3) + 16 * b;
                    if (src[b] && (MODE != M_FP4 || static_cast<size_t>(piece) * 128 + 16 * q < pitch))
                        cp_async_16(bdst + n * 128 + ((q ^ (n & 7)) << 4), src[b] + static_cast<size_t>(piece) * 128);
                }
                uint8_t* sf = slot + sf_at + r * Form<MODE>::SF + word;
                if (MODE == M_FP8) {
                    // the weight scale's UE8M0 byte, once per 32 columns
                    *reinterpret_cast<uint32_t*>(sf) = ((__float_as_uint(wsc[r]) >> 23) & 0xFFu) * 0x01010101u;
                    if (bs) cp_async_4(sf + 512, bs + 4 * piece);
                }
                if (MODE == M_FP4) {
                    const bool two = piece * KP + 128 < j.k;   // the piece's second 128 columns exist
                    if (as) {
                        cp_async_4(sf, as + 8 * piece);
                        if (two) cp_async_4(sf + 512, as + 8 * piece + 4);
                    }
                    if (bs) {
                        cp_async_4(sf + 1024, bs + 8 * piece);
                        if (two) cp_async_4(sf + 1536, bs + 8 * piece + 4);
                    }
                }
            }
            cp_async_arrive(c.full + ring.slot);
            if (MODE == M_FP8) {
                mbar_arrive(c.full + ring.slot);               // the scales stored above
                fetch(s + NP);
            }
            ring.next(c.p.slots);
        }
    }
}

// ---------------------------------------------------------------- MMA issue (one warp)
//
// The warp runs the loop as a whole and one elected lane issues: descriptors
// and counters then are warp-uniform values (issued from a loop that only one
// lane runs, an MMA cost about 200 cycles of moves, more than it takes).

struct MmaState {
    Ring ring;
    int jobs = 0, slots = 0;
    bool leader;
};

__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// wait() for a whole warp, which stays converged.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const Ctx& c) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait(bar, parity, c));
}

template <int MODE>
__device__ __forceinline__ bool issue_job(const Ctx& c, const Job& j, uint32_t tmem, uint64_t* accf, uint64_t* acce,
                                          MmaState& st) {
    const int buf = st.jobs & 1;
    if (!wait_warp(acce + buf, ((st.jobs >> 1) & 1) ^ 1u, c)) return false;
    tc_fence_after();
    const uint32_t d = tmem + buf * ACC_COLS;
    const uint32_t n = round16(__popc(__shfl_sync(0xffffffffu, j.mask, 0)) * Form<MODE>::P);
    const uint32_t idesc = MODE == M_BF16 ? make_idesc(1, 128, n) : MODE == M_FP8 ? make_idesc_mxf8(128, n)
                                                                                 : make_idesc_mxf4(n, 0);
    const uint32_t idesc2 = MODE == M_FP4 ? make_idesc_mxf4(n, 2) : idesc;
    const int p0 = __shfl_sync(0xffffffffu, j.p0, 0), p1 = __shfl_sync(0xffffffffu, j.p1, 0);
    // MXFP4: the last piece of K may be a half
    const int whole = MODE == M_FP4 ? __shfl_sync(0xffffffffu, j.k, 0) / Form<MODE>::KP : p1;
    const int row_bytes = rows_bytes<MODE>(c), sf_at = scales_at<MODE>(c);
    for (int s = p0; s < p1; s += NP) {
        if (!wait_warp(c.full + st.ring.slot, st.ring.phase, c)) return false;
        fence_proxy_async_smem();                              // the token side was copied through the generic proxy
        if (MODE != M_BF16 && st.slots >= 2) {
            // the MMAs that read this half of the scale columns two slots ago are done
            int q = st.ring.slot - 2;
            uint32_t ph = st.ring.phase;
            if (q < 0) { q += c.p.slots; ph ^= 1u; }
            if (!wait_warp(c.empty + q, ph, c)) return false;
        }
        tc_fence_after();
        uint8_t* slot = slot_at(c, st.ring.slot);
        const uint32_t sf0 = tmem + SF_COL0 + (st.slots & 1) * SF_COLS;
#pragma unroll
        for (int r = 0; r < NP; ++r) {
            if (s + r >= p1) break;
            const uint64_t a = smem_desc_k_sw128(slot + r * PIECE_BYTES);
            const uint64_t b = smem_desc_k_sw128(slot + NP * PIECE_BYTES + r * row_bytes);
            const uint32_t more = s + r > p0 ? 1u : 0u;
            const uint8_t* sf = slot + sf_at + r * Form<MODE>::SF;
            const uint32_t t = sf0 + r * (SF_COLS / NP);
            if (MODE == M_BF16) {
                if (st.leader) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma_f16(d, a + 2 * k, b + 2 * k, idesc, more | (k > 0));
                }
            } else if (MODE == M_FP8) {
                if (st.leader) {
                    tmem_cp_scales(t, sf);
                    tmem_cp_scales(t + 4, sf + 512);
#pragma unroll
                    for (int k = 0; k < 4; ++k) umma_mxf8_bs(d, a + 2 * k, b + 2 * k, idesc, t, t + 4, more | (k > 0));
                }
            } else {
                if (st.leader) {
                    tmem_cp_scales(t, sf);
                    tmem_cp_scales(t + 8, sf + 1024);
                    umma_mxf4_bs(d, a, b, idesc, t, t + 8, more);
                    umma_mxf4_bs(d, a + 2, b + 2, idesc2, t, t + 8, 1);
                    if (s + r < whole) {
                        tmem_cp_scales(t + 4, sf + 512);
                        tmem_cp_scales(t + 12, sf + 1536);
                        umma_mxf4_bs(d, a + 4, b + 4, idesc, t + 4, t + 12, 1);
                        umma_mxf4_bs(d, a + 6, b + 6, idesc2, t + 4, t + 12, 1);
                    }
                }
            }
        }
        ++st.slots;
        if (st.leader) umma_commit(c.empty + st.ring.slot);
        st.ring.next(c.p.slots);
    }
    if (st.leader) umma_commit(accf + buf);
    ++st.jobs;
    return true;
}

// ---------------------------------------------------------------- epilogue (128 threads, thread = row)

// Waits for a job's accumulator and gives body(token, value) for every token
// of the job, in ascending order.
template <int MODE, typename F>
__device__ __forceinline__ void read_job(const Ctx& c, const Job& j, uint32_t tmem, uint64_t* accf, uint64_t* acce,
                                         int& jobs, bool& ok, F&& body) {
    const int buf = jobs & 1;
    if (ok) {
        int w = 1;
        if (c.lane == 0) w = wait(accf + buf, (jobs >> 1) & 1, c);
        ok = __shfl_sync(0xffffffffu, w, 0) != 0;
    }
    ++jobs;
    if (!ok) return;
    tc_fence_after();
    const uint32_t acc = tmem + (static_cast<uint32_t>(c.warp * 32) << 16) + buf * ACC_COLS;
    uint32_t m = j.mask;
    if (Form<MODE>::P == 1) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(acc, r);
        tmem_ld_wait_regs(r);
        tc_fence_before();
        mbar_arrive(acce + buf);
#pragma unroll
        for (int i = 0; i < MAX_T; ++i) {
            if (!m) break;
            body(__ffs(m) - 1, __uint_as_float(r[i]));
            m &= m - 1;
        }
    } else {
        // five columns a token (the load reads three more)
        for (int i = 0; m; ++i, m &= m - 1) {
            uint32_t r[8];
            tmem_ld_32x32b_x8(acc + static_cast<uint32_t>(PLANES * i), r);
            tmem_ld_wait_regs(r);
            float v = __uint_as_float(r[PLANES - 1]);
#pragma unroll
            for (int q = PLANES - 2; q >= 0; --q) v += __uint_as_float(r[q]);
            body(__ffs(m) - 1, v);
        }
        tc_fence_before();
        mbar_arrive(acce + buf);
    }
}

// A tile that crosses blocks: stores this block's sums (sums[t * 128] for the
// thread's row, tokens of `mask`), and in the last of the tile's blocks to get
// here replaces them by the total over the blocks, in block order.  True where
// the sums are now the tile's.  Every epilogue thread calls it.
__device__ __forceinline__ bool combine(const Ctx& c, const Job& j, uint32_t mask, float* sums) {
    const FewParams& p = c.p;
    if (j.block0 == j.block1) return true;
    const int b = blockIdx.x;
    // a block has at most one tile it continues and one it leaves unfinished
    auto part = [&](int blk) { return p.sums + (static_cast<size_t>(blk) * 2 + (blk == j.block0)) * p.T * 128 + c.tid; };
    float* mine = part(b);
    for (uint32_t m = mask; m; m &= m - 1) {
        const int t = __ffs(m) - 1;
        __stcg(mine + t * 128, sums[t * 128]);
    }
    int* last_s = reinterpret_cast<int*>(c.smem + OFF_MISC) + 3;
    __threadfence();
    bar_epilogue();
    if (c.tid == 0) {
        uint32_t* ctr = p.ctr + CTR_TILE + j.block0;
        const bool last = atomicAdd(ctr, 1u) == static_cast<uint32_t>(j.block1 - j.block0);
        if (last) *ctr = 0;
        __threadfence();
        *last_s = last;
    }
    bar_epilogue();
    const bool last = *last_s != 0;
    bar_epilogue();                                            // the flag may be written again
    if (!last) return false;
    for (uint32_t m = mask; m; m &= m - 1) {
        const int t = __ffs(m) - 1;
        float v = 0.f;
#pragma unroll 4
        for (int blk = j.block0; blk <= j.block1; ++blk) v += __ldcg(part(blk) + t * 128);
        sums[t * 128] = v;
    }
    return true;
}

// ---------------------------------------------------------------- phase 1

// Router slices are at most 14 x 128 columns: a warp holds an expert's slice
// in registers (14 float4 a lane, one round of loads) and runs the tokens past
// it.
constexpr int SLICE_PIECES = 14;

template <int MODE>
__device__ __forceinline__ void router_and_x(const Ctx& c) {
    const FewParams& p = c.p;
    // a block has one slice of d and a share of the experts; it stages the
    // tokens' slices in the ring's memory
    const int sharers = gridDim.x / p.ks, who = blockIdx.x / p.ks, ks = blockIdx.x % p.ks;
    __nv_bfloat16* xsm = reinterpret_cast<__nv_bfloat16*>(c.smem + OFF_RING);
    if (who < sharers) {
        const int e0 = p.E * who / sharers, e1 = p.E * (who + 1) / sharers;
        const int k0 = ks * p.slice, len = min(p.slice, p.d - k0);       // multiples of 64
        const int rounds = (len + 127) / 128;                            // (zeros up to the last one's end)
        for (int i = c.tid; i < p.T * rounds * 16; i += CT) {
            const int t = i / (rounds * 16), q = i - t * rounds * 16;
            reinterpret_cast<uint4*>(xsm + t * p.slice)[q] = 8 * q < len
                ? __ldg(reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(t) * p.d + k0) + q) : make_uint4(0, 0, 0, 0);
        }
        for (int e = e0 + c.warp; e < e0 + (e1 - e0 + CW - 1) / CW * CW; e += CW) {
            float4 w[SLICE_PIECES];
            const float4* src = reinterpret_cast<const float4*>(p.W_r + static_cast<size_t>(min(e, p.E - 1)) * p.d + k0);
#pragma unroll
            for (int i = 0; i < SLICE_PIECES; ++i)
                w[i] = 32 * i + c.lane < len / 4 ? __ldg(src + 32 * i + c.lane) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (e < e0 + CW) bar_general();                              // the slices of x are there
            if (e >= e1) continue;
#pragma unroll 1
            for (int t = 0; t < p.T; ++t) {
                float acc = 0.f;
#pragma unroll
                for (int i = 0; i < SLICE_PIECES; ++i) {
                    if (i < rounds) {
                        const uint2 xv = *reinterpret_cast<const uint2*>(xsm + t * p.slice + 4 * (32 * i + c.lane));
                        acc = fmaf(__uint_as_float(xv.x << 16), w[i].x, acc);
                        acc = fmaf(__uint_as_float(xv.x & 0xFFFF0000u), w[i].y, acc);
                        acc = fmaf(__uint_as_float(xv.y << 16), w[i].z, acc);
                        acc = fmaf(__uint_as_float(xv.y & 0xFFFF0000u), w[i].w, acc);
                    }
                }
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
                if (c.lane == 0) p.part[(static_cast<size_t>(ks) * p.T + t) * p.E + e] = acc;
            }
        }
    }
    if (MODE != M_BF16) {
        const int nb = p.d / 128;
        for (int i = blockIdx.x * CW + c.warp; i < p.T * nb; i += gridDim.x * CW) {
            const int t = i / nb, b = i % nb;
            const uint2 raw = __ldg(reinterpret_cast<const uint2*>(p.x + static_cast<size_t>(t) * p.d + b * 128) + c.lane);
            store_block<MODE>(make_float4(__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u),
                                          __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xFFFF0000u)),
                              p.xq, p.xs, t, p.d, b * 128, c.lane);
        }
    }
}

// ---------------------------------------------------------------- selection

// Order-preserving key of a float, at least 1 (0 marks a taken expert).
__device__ __forceinline__ uint32_t order_key(float v) {
    const uint32_t b = __float_as_uint(v);
    return max(b & 0x80000000u ? ~b : b | 0x80000000u, 1u);
}

// Top-K, gates and the list of experts reached, by every block for itself (the
// last block also keeps the probabilities, for balance()).  The number of
// experts reached goes to the block's misc words.
__device__ __forceinline__ void select_experts(const Ctx& c) {
    const FewParams& p = c.p;
    int* idx_s = reinterpret_cast<int*>(c.smem + OFF_IDX);
    float* gate_s = reinterpret_cast<float*>(c.smem + OFF_GATE);
    uint32_t* mask_s = reinterpret_cast<uint32_t*>(c.smem + OFF_MASK);
    uint64_t* kpack_s = reinterpret_cast<uint64_t*>(c.smem + OFF_KPACK);
    int* act_s = reinterpret_cast<int*>(c.smem + OFF_ACT);
    int* misc = reinterpret_cast<int*>(c.smem + OFF_MISC);
    const bool writer = blockIdx.x == gridDim.x - 1;
    for (int t = c.warp; t < p.T; t += CW) {
        float l[8];
        uint32_t key[8];
        float top = -INFINITY;
        const float* part = p.part + static_cast<size_t>(t) * p.E;
#pragma unroll
        for (int i = 0; i < 8; ++i) l[i] = 0.f;
        // every load of a round is issued before the first is used (experts past
        // the last one read the last one's)
#pragma unroll 2
        for (int s = 0; s < p.ks; ++s) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = __ldcg(part + s * p.T * p.E + min(32 * i + c.lane, p.E - 1));
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] += v[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = 32 * i + c.lane;
            const bool in = e < p.E;
            if (in && p.logit_bias) l[i] += __ldg(p.logit_bias + e);
            key[i] = in ? order_key(p.sel_bias ? l[i] + __ldg(p.sel_bias + e) : l[i]) : 0u;
            if (!in) l[i] = -INFINITY;
            top = fmaxf(top, l[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            l[i] = expf(l[i] - top);
            sum += l[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (writer) {
            const float inv = 1.f / sum;
#pragma unroll
            for (int i = 0; i < 8; ++i) p.prob[t * 256 + 32 * i + c.lane] = l[i] * inv;
        }
        float chosen = 0.f, mine = 0.f;
        for (int k = 0; k < p.K; ++k) {
            uint32_t bk = 0, bi = 0xFFFFu;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (key[i] > bk) { bk = key[i]; bi = 32 * i + c.lane; }
            const uint32_t best = __reduce_max_sync(0xffffffffu, bk);
            const uint32_t e = __reduce_min_sync(0xffffffffu, bk == best ? bi : 0xFFFFu);
            float v = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (e == static_cast<uint32_t>(32 * i + c.lane)) { v = l[i]; key[i] = 0; }
            v = __shfl_sync(0xffffffffu, v, e & 31);
            chosen += v;
            if (c.lane == k) mine = v;
            if (c.lane == 0) idx_s[t * 16 + k] = static_cast<int>(e);
        }
        if (c.lane < p.K) gate_s[t * 16 + c.lane] = mine / chosen;
    }
    mask_s[c.tid] = 0;
    kpack_s[c.tid] = 0;
    bar_general();
    // the slots of every expert as bits (a token has at most one)
    {
        const int t = c.tid / 16, k = c.tid % 16;
        if (t < p.T && k < p.K) {
            const int e = idx_s[t * 16 + k];
            atomicOr(mask_s + e, 1u << t);
            atomicOr(reinterpret_cast<unsigned long long*>(kpack_s + e), static_cast<unsigned long long>(k) << (4 * t));
        }
    }
    bar_general();
    // one thread per expert: those within the capacity
    const int e = c.tid;
    uint32_t mask = mask_s[e];
    const int count = __popc(mask);
    reinterpret_cast<int*>(c.smem + OFF_COUNT)[e] = count;
    if (p.capacity >= 0 && count > p.capacity) {
        uint32_t keep = 0;
        int left = p.capacity;
        const uint64_t kpack = kpack_s[e];
        for (int k = 0; k < (p.slot_major ? p.K : 1); ++k)
            for (uint32_t m = mask; m && left > 0; m &= m - 1) {
                const int t = __ffs(m) - 1;
                if (!p.slot_major || (static_cast<int>(kpack >> (4 * t)) & 15) == k) { keep |= 1u << t; --left; }
            }
        mask = keep;
        mask_s[e] = keep;
    }
    const uint32_t votes = __ballot_sync(0xffffffffu, mask != 0);
    if (c.lane == 0) misc[4 + c.warp] = __popc(votes);
    bar_general();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < CW; ++w) {
        const int n = misc[4 + w];
        if (w < c.warp) base += n;
        total += n;
    }
    if (mask) act_s[base + __popc(votes & ((1u << c.lane) - 1u))] = e;
    if (c.tid == 0) misc[1] = total;
}

// The routing outputs and the balance statistics, by the token-side threads of
// the last block once they have no copies left to make.
__device__ __forceinline__ void balance(const Ctx& c) {
    const FewParams& p = c.p;
    const int i = c.tid - EPI;
    for (int s = i; s < p.T * p.K; s += EPI) {
        const int at = s / p.K * 16 + s % p.K;
        if (p.topk_idx) p.topk_idx[s] = reinterpret_cast<const int*>(c.smem + OFF_IDX)[at];
        if (p.gates) p.gates[s] = reinterpret_cast<const float*>(c.smem + OFF_GATE)[at];
    }
    float sum = 0.f;
    for (int e = i; e < p.E; e += EPI) {
        float P = 0.f;
        for (int t = 0; t < p.T; ++t) P += __ldcg(p.prob + t * 256 + e);
        P /= static_cast<float>(p.T);
        const int count = reinterpret_cast<const int*>(c.smem + OFF_COUNT)[e];
        const float f = static_cast<float>(count) / static_cast<float>(p.T * p.K);
        p.P[e] = P;
        p.f[e] = f;
        if (p.counts) p.counts[e] = count;
        sum += f * P;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    float* red = reinterpret_cast<float*>(c.smem + OFF_MISC) + 4;         // the selection's counts
    if (c.lane == 0) red[c.warp - 4] = sum;
    bar_tokens();
    if (i == 0) *p.loss = p.alpha * p.E * (red[0] + red[1] + red[2] + red[3]);
}

// ---------------------------------------------------------------- the kernel

template <int MODE>
__global__ void __launch_bounds__(THREADS, 1)
few_tokens_kernel(const __grid_constant__ FewParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint64_t* accf = full + 2 * MAX_SLOTS;
    uint64_t* acce = accf + 2;
    uint64_t* drain = acce + 2;
    int* misc = reinterpret_cast<int*>(smem + OFF_MISC);
    const Ctx c{p, smem, full, full + MAX_SLOTS, misc, static_cast<int>(threadIdx.x),
                static_cast<int>(threadIdx.x >> 5), static_cast<int>(threadIdx.x & 31)};
    if (c.tid == 0) {
        for (int i = 0; i < p.slots; ++i) {
            // expect_tx; the token side's copies and, in FP8, stores
            mbar_init(c.full + i, 1 + EPI * (MODE == M_FP8 ? 2 : 1));
            mbar_init(c.empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) { mbar_init(accf + i, 1); mbar_init(acce + i, EPI); }
        mbar_init(drain, 1);
        misc[0] = 0;
        fence_mbar_init();
    }
    if (c.warp == W_MMA) tmem_alloc<TMEM_COLS>(reinterpret_cast<uint32_t*>(misc + 2));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(misc[2]);

    if (c.warp == W_TMA) {
        if (c.lane == 0) {
            tma_prefetch_desc(&p.w1);
            tma_prefetch_desc(&p.w2);
            if (p.S) { tma_prefetch_desc(&p.ws1); tma_prefetch_desc(&p.ws2); }
        }
        __syncthreads();                                        // the experts are selected
        const int n_active = misc[1];
        Ring ring;
        bool ok = *c.abort_flag == 0;
        Job j;
#pragma unroll 1
        for (int phase = 2; phase <= 3; ++phase)
            for (Jobs<MODE> jobs(c, phase, n_active); ok && jobs.next(j);)
                ok = load_weights<MODE>(c, j, phase == 2 ? (j.shared ? &p.ws1 : &p.w1) : (j.shared ? &p.ws2 : &p.w2), ring);
        // a block that gave up leaves its copies the time to land before it
        // gives its memory back (their barriers may never complete, since the
        // token side stopped arriving)
        if (!ok && c.lane == 0) {
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < kDrainNs) {}
        }
        __syncwarp();
    } else if (c.warp == W_MMA) {
        __syncthreads();
        const int n_active = misc[1];
        MmaState st;
        st.leader = elect_one();
        bool ok = *c.abort_flag == 0;
        Job j;
#pragma unroll 1
        for (int phase = 2; phase <= 3; ++phase)
            for (Jobs<MODE> jobs(c, phase, n_active); ok && jobs.next(j);) ok = issue_job<MODE>(c, j, tmem, accf, acce, st);
        if (!ok && st.slots && st.leader) {
            umma_commit(drain);
            volatile int no_abort = 0;
            mbar_wait_bounded(drain, 0, &no_abort, nullptr, kDrainNs);
        }
        __syncwarp();
    } else {
        router_and_x<MODE>(c);
        grid_barrier(p.ctr, 0, p.status, c.abort_flag, c.tid);
        select_experts(c);
        fence_proxy_async_smem();                               // phase 1 used the ring's memory
        __syncthreads();
        const int n_active = misc[1];
        const int* idx_s = reinterpret_cast<const int*>(smem + OFF_IDX);
        const float* gate_s = reinterpret_cast<const float*>(smem + OFF_GATE);
        const uint32_t* mask_s = reinterpret_cast<const uint32_t*>(smem + OFF_MASK);
        const int slots_h = p.T * p.K;                          // rows of routed h
        const size_t h_shared = static_cast<size_t>(slots_h) * p.dff;
        float* sums = reinterpret_cast<float*>(smem + OFF_OUT) + c.tid;            // epilogue: [t * 128]
        Ring ring;
        int jobs_read = 0;
        bool ok = *c.abort_flag == 0;
#pragma unroll 1
        for (int phase = 2; phase <= 3; ++phase) {
            const bool third = phase == 3;
            if (third) {
                grid_barrier(p.ctr, 1, p.status, c.abort_flag, c.tid);
                if (MODE != M_BF16) {
                    // h in operand form, a warp per 128 values that phase 3
                    // reads; a slot over the capacity has none
                    constexpr int P = Form<MODE>::P;
                    const int nr = p.dff / 128, ns = p.dffs / 128;
                    const int routed = slots_h * nr, blocks = routed + p.S * p.T * ns;
                    uint8_t* hq_shared = p.hq + h_shared * P / (MODE == M_FP4 ? 2 : 1);
                    uint8_t* hs_shared = p.hs + (MODE == M_FP4 ? h_shared * P / 32 : h_shared / 128 * 4);
                    for (int i = blockIdx.x * CW + c.warp; i < blocks; i += gridDim.x * CW) {
                        const bool sh = i >= routed;
                        const int u = sh ? i - routed : i, nb = sh ? ns : nr, row = u / nb, col = u % nb * 128;
                        const int t = row / p.K;
                        if (!sh && !(mask_s[idx_s[t * 16 + row - t * p.K]] >> t & 1u)) continue;
                        const int k = sh ? p.dffs : p.dff;
                        const float4 v = __ldcg(reinterpret_cast<const float4*>(
                            p.h32 + (sh ? h_shared : 0) + static_cast<size_t>(row) * k + col) + c.lane);
                        store_block<MODE>(v, sh ? hq_shared : p.hq, sh ? hs_shared : p.hs, row, k, col, c.lane);
                    }
                    grid_barrier(p.ctr, 2, p.status, c.abort_flag, c.tid);
                }
                ok = ok && *c.abort_flag == 0;
            }
            if (c.warp >= 4) {
                load_tokens<MODE>(c, phase, n_active, h_shared, ring, ok);
                if (third && blockIdx.x == gridDim.x - 1) balance(c);
                continue;
            }
            bool begins = true;
            Job j;
            for (Jobs<MODE> jobs(c, phase, n_active); jobs.next(j);) {
                if (begins) for (int t = 0; t < p.T; ++t) sums[t * 128] = 0.f;
                begins = j.ends;
                const int row = j.row0 + c.tid;
                const bool in = row < j.n;
                // phase 3: the block with a matrix's first piece adds its bias
                const float* biases = third ? (j.shared ? p.bs2 : p.b2) : (j.shared ? p.bs1 : p.b1);
                const float bias = in && (!third || j.p0 == 0) ? __ldg(biases + static_cast<size_t>(j.mat) * j.n + row) : 0.f;
                const bool gated = third && !j.shared;
                const float inner = third ? bias : 0.f;
                read_job<MODE>(c, j, tmem, accf, acce, jobs_read, ok, [&](int t, float v) {
                    const float g = gated ? gate_s[t * 16 + (static_cast<int>(j.kpack >> (4 * t)) & 15)] : 1.f;
                    sums[t * 128] = fmaf(g, v + inner, sums[t * 128]);
                });
                const uint32_t tokens = third ? (1u << p.T) - 1u : j.mask;
                if (!j.ends || !combine(c, j, tokens, sums) || !in || !ok) continue;
                const size_t base = j.shared ? h_shared : 0;
                for (uint32_t m = tokens; m; m &= m - 1) {
                    const int t = __ffs(m) - 1;
                    float v = sums[t * 128];
                    if (!third) {
                        const float h = silu_fast(v + bias);
                        const size_t at = base + static_cast<size_t>(h_row(c, j, t)) * j.n + row;
                        if (MODE == M_BF16) reinterpret_cast<__nv_bfloat16*>(p.hq)[at] = __float2bfloat16_rn(h);
                        else p.h32[at] = h;
                        continue;
                    }
                    const size_t at = static_cast<size_t>(t) * p.d + row;
                    if (p.passthrough) {
                        for (int k = 0; k < p.K; ++k)
                            if (!(mask_s[idx_s[t * 16 + k]] >> t & 1u))
                                v = fmaf(gate_s[t * 16 + k], __bfloat162float(p.x[at]), v);
                    }
                    p.out[at] = __float2bfloat16_rn(v);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    // the last block to leave zeroes the counters for the next launch
    if (c.tid == 0) {
        __threadfence();
        if (atomicAdd(p.ctr + CTR_EXIT, 1u) == gridDim.x - 1) {
            for (int i = 0; i < CTR_WORDS; ++i) p.ctr[i] = 0;
            __threadfence();
        }
    }
    if (c.warp == W_MMA) {
        tc_fence_after();
        tmem_dealloc<TMEM_COLS>(tmem);
    }
}

size_t align256(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

struct FewLayout {
    size_t ctr, part, prob, xq, xs, h32, hq, hs, sums, total;
};

// blocks: as many as can find work, at most one per SM
struct FewPlan {
    int blocks, ks, slice;
};

FewPlan few_plan(const Dims& dm, int sms) {
    FewPlan f;
    if (sms > MAX_BLOCKS) sms = MAX_BLOCKS;
    // a block per slot of weights that the most experts reached would have
    const int kp = dm.dtype == MOE_BF16 ? Form<M_BF16>::KP : dm.dtype == MOE_MXFP4 ? Form<M_FP4>::KP : Form<M_FP8>::KP;
    auto slots = [&](long long rows, long long k) { return (rows + 127) / 128 * ((k + NP * kp - 1) / (NP * kp)); };
    const long long reached = dm.T * dm.K < dm.E ? dm.T * dm.K : dm.E;
    const long long s2 = reached * slots(dm.dff, dm.d) + dm.S * slots(dm.dffs, dm.d);
    const long long s3 = reached * slots(dm.d, dm.dff) + dm.S * slots(dm.d, dm.dffs);
    const long long most = s2 > s3 ? s2 : s3;
    f.blocks = most < sms ? static_cast<int>(most) : sms;
    // router: slices of d (multiples of 128 columns), as many as give each
    // block at most one expert a warp
    static_assert(MAX_T * 128 * SLICE_PIECES * 2 <= RING_BYTES, "the staged slice of x fits the ring");
    int want = f.blocks * CW / dm.E;
    if (want > 16) want = 16;
    if (want > f.blocks) want = f.blocks;
    if (want < 1) want = 1;
    const int pieces = (dm.d + 127) / 128;
    int per = (pieces + want - 1) / want;
    if (per > SLICE_PIECES) per = SLICE_PIECES;
    f.slice = 128 * per;
    f.ks = (pieces + per - 1) / per;
    if (f.blocks < f.ks) f.blocks = f.ks;
    return f;
}

FewLayout few_layout(const Dims& dm) {
    FewLayout L{};
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off = align256(off + bytes); return o; };
    const bool q = dm.dtype != MOE_BF16, fp4 = dm.dtype == MOE_MXFP4;
    const size_t h = static_cast<size_t>(dm.T) * dm.K * dm.dff + static_cast<size_t>(dm.S) * dm.T * dm.dffs;
    const size_t x = static_cast<size_t>(dm.T) * dm.d;
    // bytes of n elements in operand form, and of their scales
    auto form = [&](size_t n) { return fp4 ? n * PLANES / 2 : q ? n : 2 * n; };
    auto scales = [&](size_t n) { return fp4 ? n * PLANES / 32 : q ? n / 128 * 4 : 0; };
    take(256);                                              // status word
    L.ctr = take((CTR_TILE + MAX_BLOCKS) * 4);
    // slices are at least 128 columns long, whatever the device's size
    L.part = take(static_cast<size_t>((dm.d + 127) / 128) * dm.T * dm.E * 4);
    L.prob = take(static_cast<size_t>(dm.T) * 256 * 4);
    L.xq = take(q ? form(x) : 0);
    L.xs = take(scales(x));
    L.h32 = take(q ? h * 4 : 0);
    L.hq = take(form(h));
    L.hs = take(scales(h));
    L.sums = take(static_cast<size_t>(MAX_BLOCKS) * 2 * dm.T * 128 * 4);
    L.total = off;
    return L;
}

template <int MODE>
cudaError_t launch_mode(FewParams& p, int blocks, cudaStream_t st) {
    constexpr int rows_max = round16(MAX_T * Form<MODE>::P) * 128;
    static_assert(RING_BYTES / (NP * (PIECE_BYTES + rows_max + Form<MODE>::SF)) >= 3, "two slots of MMAs in flight");
    p.slot_bytes = NP * (PIECE_BYTES + round16(p.T * Form<MODE>::P) * 128 + Form<MODE>::SF);
    p.slots = RING_BYTES / p.slot_bytes < MAX_SLOTS ? RING_BYTES / p.slot_bytes : MAX_SLOTS;
    auto kernel = few_tokens_kernel<MODE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_ALLOC);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_ALLOC;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    count_launches(1);
    e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

size_t few_ws_bytes(const Dims& dm) { return few_layout(dm).total; }

cudaError_t launch_few(const Dims& dm, const FewArgs& a, void* ws, cudaStream_t st) {
    FewParams p;
    std::memset(&p, 0, sizeof(p));
    const FewLayout L = few_layout(dm);
    uint8_t* w = static_cast<uint8_t*>(ws);
    const FewPlan plan = few_plan(dm, device_sm_count());
    p.x = static_cast<const __nv_bfloat16*>(a.x);
    p.W_r = a.W_r;
    p.logit_bias = dm.bias_mode == MOE_BIAS_LOGITS ? a.logit_bias : nullptr;
    p.sel_bias = dm.bias_mode == MOE_BIAS_SELECTION ? a.logit_bias : nullptr;
    p.w1s = a.W1_scales;
    p.w2s = a.W2_scales;
    p.ws1s = a.Ws1_scales;
    p.ws2s = a.Ws2_scales;
    p.b1 = a.b1;
    p.b2 = a.b2;
    p.bs1 = a.bs1;
    p.bs2 = a.bs2;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.f = a.f;
    p.P = a.P;
    p.loss = a.loss;
    p.topk_idx = a.topk_idx;
    p.gates = a.gates;
    p.counts = a.counts;
    p.status = reinterpret_cast<int32_t*>(w);
    p.ctr = reinterpret_cast<uint32_t*>(w + L.ctr);
    p.part = reinterpret_cast<float*>(w + L.part);
    p.prob = reinterpret_cast<float*>(w + L.prob);
    p.xq = dm.dtype == MOE_BF16 ? const_cast<uint8_t*>(static_cast<const uint8_t*>(a.x)) : w + L.xq;
    p.xs = w + L.xs;
    p.h32 = reinterpret_cast<float*>(w + L.h32);
    p.hq = w + L.hq;
    p.hs = w + L.hs;
    p.sums = reinterpret_cast<float*>(w + L.sums);
    p.alpha = dm.alpha;
    p.T = dm.T;
    p.d = dm.d;
    p.E = dm.E;
    p.K = dm.K;
    p.dff = dm.dff;
    p.S = dm.S;
    p.dffs = dm.dffs;
    p.capacity = dm.capacity;
    p.slot_major = dm.slot_major;
    p.passthrough = dm.passthrough;
    p.ks = plan.ks;
    p.slice = plan.slice;
    const int elem = dm.dtype == MOE_BF16 ? 2 : 1;
    const int div = dm.dtype == MOE_MXFP4 ? 2 : 1;           // elements of K per map element
    if (!encode_tma_3d(&p.w1, a.W1, dm.E, dm.dff, dm.d / div, elem, 128) ||
        !encode_tma_3d(&p.w2, a.W2, dm.E, dm.d, dm.dff / div, elem, 128))
        return cudaErrorInvalidValue;
    if (dm.S > 0 && (!encode_tma_3d(&p.ws1, a.Ws1, dm.S, dm.dffs, dm.d / div, elem, 128) ||
                     !encode_tma_3d(&p.ws2, a.Ws2, dm.S, dm.d, dm.dffs / div, elem, 128)))
        return cudaErrorInvalidValue;
    if (dm.dtype == MOE_BF16) return launch_mode<M_BF16>(p, plan.blocks, st);
    if (dm.dtype == MOE_FP8_E4M3_BLOCK) return launch_mode<M_FP8>(p, plan.blocks, st);
    return launch_mode<M_FP4>(p, plan.blocks, st);
}

}  // namespace moe
