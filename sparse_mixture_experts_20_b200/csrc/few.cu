// The whole layer for a few tokens (T <= 16) in one persistent kernel.
//
// Decoding a few tokens is bound by the bytes of the experts they reach, so
// the kernel is a stream of weight rows through every SM that nothing
// interrupts: pieces of 128 weight rows x 128 bytes go by TMA into a ring in
// shared memory, and tcgen05 multiplies them in place, the weights as the
// 128-row operand and the tokens as a narrow one.  No thread touches a weight,
// and what a slot of the ring needs of the tokens is one or two bulk copies,
// because phases 1 and 2 write x and h as the image that the tensor core reads.
// One block per SM, launched cooperatively; the phases are separated by grid
// barriers, and since weights do not depend on what the second waits for, the
// ring keeps filling across it:
//   1  router logits: (expert, slice of d) dot products in fp32, partial sums
//      per slice; the image of x;
//   -- barrier; every block then selects the top-K of all tokens for itself
//      (slices added in order) and builds the list of experts reached;
//   2  h = SiLU(W1 x + b1), into its image: a tile's 128 rows are 128 columns
//      of h, which FP8 and MXFP4 scale together or in fours;
//   -- barrier;
//   3  out = sum over the experts of gate * (W2 h + b2), shared experts
//      included.
// Phases 2 and 3 are one sequence each of tiles of 128 result rows (phase 2:
// of every expert's W1; phase 3: of the output, through every expert's W2),
// each a run of slots (two pieces of K), cut into a large share for every
// block and, where that is long, small ones that the blocks take as they get to
// them: SMs do not stream at the same speed (on B200 a quarter of them about
// 12 % slower, GPC by GPC).  A tile that crosses a border between shares is
// summed from the shares' parts, in order, by whichever block finishes last:
// who takes a share changes nothing in the sums.
//
// Operand forms (products exact, sums in fp32):
//   bf16   weights, x and h in bf16 (kind::f16): h is rounded as the ordinary
//          layer rounds it, since both operands of an MMA have one type (error
//          against fp64 2.3e-3; with h in fp32 it would be the output's 1.6e-3);
//   FP8    e4m3 (kind::mxf8f6f4.block_scale); x and h quantised to e4m3 per 128
//          columns; all scales are powers of two and go to the tensor core.  A
//          tile's weight scale is one number for 128 columns of K: tensor
//          memory keeps eight "uniform" sets of scale columns, by exponent
//          modulo 8, and an MMA names the one it needs;
//   MXFP4  packed E2M1 with its E8M0 scales (kind::mxf4.block_scale), which lie
//          tiled in the order that tcgen05.cp reads.  x and h are
//          fixed point per 32 columns: split into five E2M1 planes,
//          each the nearest E2M1 value of what the planes before it left, at
//          scales s, s/4, s/32, s/256, s/2048.  A plane's remainder is at most
//          half of the step at its largest magnitude (1, then 1/2 of the next
//          plane's unit), so the five stand for the value to within s / 4096
//          <= amax / 12288.  A plane whose scale would be below 2^-127 holds
//          nothing, which leaves an error of at most 2^-126 (the first plane's
//          at scale 2^-126).  A token is then five columns, which the tensor
//          core has to spare.
//
// Per block (352 threads):
//   warps 0..7  phase 1 and selection; warps 0..3 the epilogues
//               (thread = row);
//   warp 8      plans the jobs of the block's shares, and loads weights and
//               their scales;
//   warp 9      MMA issue;          warp 10  loads the tokens' images.
// The weights stream past L2, and the code with them unless they are loaded
// evict-first (306 -> 294 us for sixteen tokens in MXFP4); even so a phase's
// first instructions cost as much as its first weights.  The role loops
// therefore run both phases through the same code (measured: 172 KB of code
// took 10 us to select the experts of one token and 7 us from there to the
// first weights).
// Measured (7168 x 2048 experts, 256 of them, top-8 and one shared): MXFP4 one
// token 43 us, sixteen 279 to 298 (1.62 GB, 5.4 to 5.8 TB/s); FP8 61 and 474 to
// 499 us (3.04 GB, 6.1 to 6.4 TB/s); bf16, eight tokens, 8 experts of 4096 x
// 14336, 290 to 295 us (1.69 GB, 5.8 TB/s).  The copy rate of the same GPUs is
// 6.5 TB/s.
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
constexpr int W_LOAD = 8, W_MMA = 9, W_TOKENS = 10;
constexpr int THREADS = CT + 96;
constexpr int EPI = 128;                       // epilogue threads
constexpr int NP = 2;                          // pieces per slot
constexpr int MAX_SLOTS = 5, PIECE_BYTES = 16384;
constexpr int MAX_T = MOE_FEW_MAX_TOKENS;
constexpr int MAX_BLOCKS = 160;                // SMs used
constexpr int SMALL = 8, SHARES = 1 + SMALL;   // shares of a phase per block, at most: one large, the others small
constexpr int JOBS = 4, JOB_PIECES = 64;       // jobs announced within a block; pieces of a job
constexpr int PLANES = 5;                      // MXFP4: columns per token
constexpr int SLICE_PIECES = 14;               // router: a slice of d has at most 14 x 128 columns
constexpr uint32_t ACC_COLS = 96, SFB_COL0 = 2 * ACC_COLS, SFB_COLS = 16, SFA_COL0 = SFB_COL0 + 2 * SFB_COLS;
constexpr uint32_t TMEM_COLS = 256;            // 2 accumulators; 2 slots of token scales; weight scales (32 columns)
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr uint64_t kDrainNs = 200000000ull;

// A job: a run of slots of one tile and one matrix: pieces p0 .. p1 - 1 of K
// (128 bytes of every row each) of rows row0 .. row0 + 127, for the tokens of
// `mask`.  Column c of the operand is token c / P (phase 2: of all; phase 3:
// the c / P-th of mask).
struct Job {
    int shared;                  // 1: shared expert
    int mat, row0;
    int n, k;                    // the matrix: n rows of k columns
    int p0, p1;                  // -1: the phase is over
    uint32_t mask;
    uint64_t kpack;              // routed: the tokens' slots, 4 bits each
    int ends;                    // the share's last job of this tile
    int share, share0, share1;   // this share, and the first and last with slots of the tile
    int small0, smalls;          // and small shares of the tile alone, from small0 on
    int base8;                   // phase 3: first row of the expert's image, in units of 8
    int rank;                    // phase 3: its place among the experts reached (shared: its number)
};

constexpr int OFF_IDX = 0;                                     // [16][16] int
constexpr int OFF_GATE = OFF_IDX + MAX_T * 16 * 4;             // [16][16] float
constexpr int OFF_MASK = OFF_GATE + MAX_T * 16 * 4;            // [256] tokens kept, per expert
constexpr int OFF_KPACK = OFF_MASK + 256 * 4;                  // [256] 4 bits per token: its slot
constexpr int OFF_ACT = OFF_KPACK + 256 * 8;                   // [256] experts reached, ascending
constexpr int OFF_COUNT = OFF_ACT + 256 * 4;                   // [256] slots that name the expert
constexpr int OFF_BASE = OFF_COUNT + 256 * 4;                  // [256] per expert: base8 | rank << 16
constexpr int OFF_OUT = OFF_BASE + 256 * 4;                    // [16][128] fp32 sums of a tile
constexpr int OFF_UNI = OFF_OUT + MAX_T * 128 * 4;             // [512] a uniform set of weight scales, on its way
constexpr int OFF_JOBS = OFF_UNI + 512;                        // [JOBS] Job
constexpr int OFF_JOBSC = OFF_JOBS + JOBS * static_cast<int>(sizeof(Job));     // [JOBS][64] FP8: weight scales, UE8M0
constexpr int OFF_BAR = OFF_JOBSC + JOBS * JOB_PIECES;         // full, empty [MAX_SLOTS]; accf, acce [2]; drain; jobs' full, empty
constexpr int N_BARS = 2 * MAX_SLOTS + 5 + 2 * JOBS;
constexpr int OFF_MISC = OFF_BAR + N_BARS * 8;                 // abort flag, n_active, tmem address, last flag, 8 warp counts, 8 warp sums
constexpr int OFF_RING = (OFF_MISC + 96 + 1023) & ~1023;
constexpr int RING_BYTES = 207 * 1024;
constexpr int SMEM_ALLOC = OFF_RING + RING_BYTES + 1024;
static_assert(SMEM_ALLOC <= 227 * 1024, "shared memory budget");
static_assert(OFF_KPACK % 8 == 0 && OFF_BAR % 8 == 0 && OFF_JOBS % 8 == 0 && sizeof(Job) % 8 == 0 && OFF_UNI % 16 == 0,
              "alignment");
static_assert(SFA_COL0 + 32 <= TMEM_COLS && PLANES * MAX_T + 3 <= ACC_COLS, "tensor memory budget");

// grid-wide counters in the workspace, zero between launches
enum { CTR_BAR = 0, CTR_EXIT = 2, CTR_ABORT = 3, CTR_SHARE = 4, CTR_WORDS = 6, CTR_TILE = 64 };

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
    float* part;                  // (ks, T, E rounded up to 4) partial logits
    float* prob;                  // (T, 256) softmax of the logits
    uint8_t *xq, *xs;             // image of x: rows, scales
    uint8_t *hq, *hs;             // image of h, routed
    uint8_t *hqs, *hss;           // image of h, shared
    float* sums;                  // (shares, 2, T, 128) parts of tiles that cross shares
    float alpha;
    int T, d, E, K, dff, S, dffs, capacity, slot_major, passthrough;
    int e4;                       // E rounded up to 4
    int ks, slice;                // router slices of d and their length
    int slots, slot_bytes;        // ring
};

enum { M_BF16 = 0, M_FP8 = 1, M_FP4 = 2 };

// KP: elements of K in a piece (128 bytes of a weight row); P: columns per
// token; SFB, SFA: bytes of the tokens' and the weights' scales per piece
template <int MODE> struct Form;
template <> struct Form<M_BF16> { static constexpr int KP = 64, P = 1, SFB = 0, SFA = 0; };
template <> struct Form<M_FP8> { static constexpr int KP = 128, P = 1, SFB = 512, SFA = 0; };
template <> struct Form<M_FP4> { static constexpr int KP = 256, P = PLANES, SFB = 1024, SFA = 1024; };

__host__ __device__ constexpr int round16(int v) { return (v + 15) & ~15; }
// Rows of an image for n tokens, in units of 8 (1024 bytes a piece).
template <int MODE> __host__ __device__ constexpr int rows8(int n) { return (n * Form<MODE>::P + 7) / 8; }
// Pieces of k columns, counted in whole slots.
template <int MODE> __host__ __device__ constexpr int slots_of(int k) { return (k + NP * Form<MODE>::KP - 1) / (NP * Form<MODE>::KP); }
template <int MODE> __host__ __device__ constexpr int pieces_of(int k) { return NP * slots_of<MODE>(k); }

__device__ __forceinline__ void bar_general() { asm volatile("bar.sync 1, %0;" :: "n"(CT) : "memory"); }
__device__ __forceinline__ void bar_epilogue() { asm volatile("bar.sync 2, %0;" :: "n"(EPI) : "memory"); }
// The epilogue warps agree: true if every one of them is ok.
__device__ __forceinline__ bool all_ok(bool ok) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.red.and.pred q, 2, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(static_cast<uint32_t>(ok)), "n"(EPI) : "memory");
    return r != 0;
}
__device__ __forceinline__ void bar_upper() { asm volatile("bar.sync 3, %0;" :: "n"(EPI) : "memory"); }       // warps 4..7
// The general warps and the token loader: what phase 2 or 3 reads is in memory.
__device__ __forceinline__ void bar_tokens_ready() { asm volatile("bar.sync 4, %0;" :: "n"(CT + 32) : "memory"); }

// Orders generic-proxy writes of global memory with async-proxy (bulk copy)
// reads of it: by the writer before the barrier, by the reader after it.
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" :: "r"(smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 :: "r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

// Loads of weights, which a call reads once: first to leave L2, so that the
// code, the router and the images stay there.
__device__ __forceinline__ uint64_t evict_first_policy() {
    uint64_t v;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(v));
    return v;
}

__device__ __forceinline__ void load_weights(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1, int c2,
                                             uint64_t policy) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
                 " [%0], [%1, {%3, %4, %5}], [%2], %6;"
                 :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2),
                    "l"(policy) : "memory");
}

__device__ __forceinline__ void load_scales(void* dst, const void* src, uint32_t bytes, uint64_t* bar, uint64_t policy) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
                 :: "r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy) : "memory");
}

__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(dst)), "l"(src) : "memory");
}

__device__ __forceinline__ void add_release(uint32_t* p) {
    asm volatile("red.release.gpu.global.add.u32 [%0], 1;" :: "l"(p) : "memory");
}

__device__ __forceinline__ uint32_t add_acq_rel(uint32_t* p) {
    uint32_t v;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

// ---------------------------------------------------------------- images of x and h
//
// Rows: per piece, the columns' rows of 128 bytes, as many groups of 8 as the
// tokens need, 16-byte chunk q of row n at chunk q ^ (n mod 8) (the 128-byte
// swizzle).  Scales: per 128 columns of K, 512 bytes with column n's word (the
// UE8M0 bytes of its four blocks of 32) at 16 (n mod 32) + 4 (n div 32).

// Four consecutive values a lane, 128 in all, of column block `col` (a
// multiple of 128), for the c-th token of an image whose pieces have r8 groups
// of rows.
template <int MODE>
__device__ __noinline__ void store_block(float4 v4, uint8_t* rows, uint8_t* scales, int r8, int c, int col, int lane) {
    float v[4] = {v4.x, v4.y, v4.z, v4.w};
    // byte `at` of row n of the piece that has it
    auto place = [&](int n, int at) {
        return rows + (static_cast<size_t>(at >> 7) * r8 + (n >> 3)) * 1024 + (n & 7) * 128 +
               ((((at >> 4) & 7) ^ (n & 7)) << 4) + (at & 15);
    };
    auto word = [&](int n) { return scales + static_cast<size_t>(col / 128) * 512 + 16 * (n & 31) + 4 * (n >> 5); };
    if (MODE == M_BF16) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *reinterpret_cast<uint2*>(place(c, 2 * (col + 4 * lane))) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    } else if (MODE == M_FP8) {
        // as the dispatch quantiser: fmaxf does not count a NaN
        float a = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) a = fmaxf(a, fabsf(v[j]));
        const uint32_t m = __reduce_max_sync(0xffffffffu, __float_as_uint(a));
        const float sc = pow2_scale_448(__uint_as_float(m)), inv = inv_pow2(sc);
        const uint32_t lo = f32x2_to_e4m3x2(v[0] * inv, v[1] * inv), hi = f32x2_to_e4m3x2(v[2] * inv, v[3] * inv);
        *reinterpret_cast<uint32_t*>(place(c, col + 4 * lane)) = lo | (hi << 16);
        if (lane == 0) *reinterpret_cast<uint32_t*>(word(c)) = (__float_as_uint(sc) >> 23) * 0x01010101u;
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
            const int n = c * PLANES + pl;
            *reinterpret_cast<uint16_t*>(place(n, col / 2 + 2 * lane)) = static_cast<uint16_t>(codes);
            if ((lane & 7) == 0) word(n)[lane / 8] = static_cast<uint8_t>(b == 255u ? 255 : max(e, 0));
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

// wait() for a whole warp, which stays converged.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, const Ctx& c) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    return __all_sync(0xffffffffu, wait(bar, parity, c));
}

// The general warps of all blocks.  Writes before it are visible to reads
// (through L2) after it: the block's barrier orders them before the release,
// the acquire before the block's next one (a fence on either side of the
// atomic took 0.3 us more).
__device__ __noinline__ void grid_barrier(uint32_t* ctrs, int which, int32_t* status, volatile int* abort_flag, int tid) {
    bar_general();
    if (tid == 0) {
        uint32_t* ctr = ctrs + CTR_BAR + which;
        add_release(ctr);
        if (*abort_flag) atomicExch(ctrs + CTR_ABORT, 1u);
        uint64_t t0 = 0;
#pragma unroll 1
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
    }
    bar_general();
}

// ---------------------------------------------------------------- jobs

// Place of token t among the columns of its expert's image of h.
__device__ __forceinline__ int column_of(const Job& j, int t) { return __popc(j.mask & ((1u << t) - 1u)); }

// The shares of a phase's slots and their jobs (planning warp).  Phase 2:
// matrix by matrix, its tiles, their slots of K = d.  Phase 3: tile by tile,
// the shared experts' slots, then those of the experts reached.
//
// Fewer than 64 slots a block: equal shares, none without slots (the join of a
// further share costs more than it evens out); in phase 2 of whole tiles, which
// need no join, where that leaves no block more than 1/16 over its share (one
// token: MXFP4 42.8 us, 45.4 without that rule; FP8 60.8 and 63.0).  Else phase
// 2 has three quarters in a large share per block and the rest, at the end of
// the sequence, in small ones of 16 slots or more.  Phase 3 has few tiles, and
// one cut into many shares would be long to add up: there the last eighth of
// every tile is small shares of its own, of 10 slots or more (sixteen tokens:
// MXFP4 279 us, FP8 474; with 12 and 10 slots 278 and 478, with 16 and 14 283
// and 472, with 8 and 7 slower by 14 and 4).
template <int MODE>
struct Plan {
    const Ctx& c;
    bool third;           // phase 3
    int share, shares, at, end;
    int lead;             // phase 2: slots of the large shares, one per block (0: none)
    int each, extra;      // slots of the equal shares; the first `extra` have one more
    int ss, sr;           // slots of a shared, a routed matrix per tile
    int ts, tr;           // phase 2: tiles of a shared, a routed matrix
    int head, tail, q;    // phase 3: a tile's slots in equal shares and in q small ones
    int equal;            // phase 3: number of equal shares
    int rest = 0;         // phase 2, whole tiles: tiles of the last share, if fewer
    __device__ __forceinline__ Plan(const Ctx& c_, int phase, int n_active) : c(c_), third(phase == 3) {
        const FewParams& p = c.p;
        const int blocks = gridDim.x;
        ss = slots_of<MODE>(third ? p.dffs : p.d);
        sr = slots_of<MODE>(third ? p.dff : p.d);
        ts = third ? 1 : (p.dffs + 127) / 128;
        tr = third ? 1 : (p.dff + 127) / 128;
        at = end = 0;
        lead = q = tail = 0;
        head = 1;
        if (!third) {
            const int tiles = p.S * ts + n_active * tr, all = tiles * sr, per = all / blocks;
            const int most = (tiles + blocks - 1) / blocks;    // tiles of a block, whole ones
            equal = 0;
            lead = per < 64 ? 0 : 3 * per / 4;
            if (!lead && 16 * most * blocks <= 17 * tiles) {
                shares = tiles / most;
                each = most * sr;
                extra = 0;
                // (the rest of the tiles, fewer than a share's, go to a last share)
                rest = tiles - shares * most;
                if (rest) ++shares;
            } else {
                const int others = lead ? blocks * max(1, min(SMALL, (per - lead) / 16)) : min(blocks, all);
                shares = others + (lead ? blocks : 0);
                each = (all - blocks * lead) / others;
                extra = all - blocks * lead - each * others;
            }
        } else {
            const int tiles = (p.d + 127) / 128, tile = p.S * ss + n_active * sr;
            // (with more tiles than blocks a share would have several tiles of
            // which parts are elsewhere, and a share has room for one it begins)
            if (tiles <= blocks && tiles * tile / blocks >= 64) {
                tail = tile / 8;
                q = min(tail / 10, min(SMALL * blocks / tiles, (4 * blocks + tiles - 1) / tiles));
                if (q < 1) q = tail = 0;
            }
            head = tile - tail;
            equal = min(blocks, tiles * head);
            each = tiles * head / equal;
            extra = tiles * head - each * equal;
            shares = equal + tiles * q;
        }
    }
    __device__ __forceinline__ void take(int s) {
        share = s;
        const int blocks = gridDim.x;
        if (third && s >= equal) {
            const int i = (s - equal) % q;
            at = tail * i / q;
            end = tail * (i + 1) / q;
        } else if (!third && lead && s < blocks) {
            at = s * lead;
            end = at + lead;
        } else {
            const int v = lead ? s - blocks : s;
            at = blocks * lead + v * each + min(v, extra);
            end = rest && s == shares - 1 ? at + rest * sr : at + each + (v < extra ? 1 : 0);
        }
    }
    // the share that has slot u (phase 3: of the equal ones)
    __device__ __forceinline__ int share_of(int u) const {
        const int blocks = gridDim.x;
        if (u < blocks * lead) return u / lead;
        u -= blocks * lead;
        const int v = u - extra * (each + 1);
        return (lead ? blocks : 0) + (v < 0 ? u / (each + 1) : extra + v / each);
    }
    // The share's next job; false at its end.
    __device__ __forceinline__ bool next(Job& j) {
        if (at >= end) return false;
        const FewParams& p = c.p;
        // u: slot of the tile (phase 3) or of the sequence; first .. last: the tile's slots of it
        int u = at, first = 0, left = end - at, tile = 0;
        if (third) {
            if (share >= equal) {
                tile = (share - equal) / q;
                u += head;
            } else {
                tile = u / head;
                first = tile * head;
                u -= first;
                left = min(left, head - u);
            }
            j.row0 = tile * 128;
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
        const int n = min(min(per - s0, left), JOB_PIECES / NP);
        j.mat = j.shared ? m : reinterpret_cast<const int*>(c.smem + OFF_ACT)[m];
        j.mask = j.shared ? (1u << p.T) - 1u : reinterpret_cast<const uint32_t*>(c.smem + OFF_MASK)[j.mat];
        j.kpack = j.shared ? 0 : reinterpret_cast<const uint64_t*>(c.smem + OFF_KPACK)[j.mat];
        const int base = j.shared ? 0 : reinterpret_cast<const int*>(c.smem + OFF_BASE)[j.mat];
        j.base8 = j.shared ? m * rows8<MODE>(p.T) : base & 0xFFFF;
        j.rank = j.shared ? m : base >> 16;
        const int inner = j.shared ? p.dffs : p.dff;
        j.n = third ? p.d : inner;
        j.k = third ? inner : p.d;
        j.p0 = s0 * NP;
        j.p1 = min((s0 + n) * NP, (j.k + Form<MODE>::KP - 1) / Form<MODE>::KP);
        at += n;
        j.ends = at == end || (third ? n == left : at == first + per);
        j.share = share;
        const int f = third ? tile * head : first;
        j.share0 = share_of(f);
        j.share1 = share_of(f + (third ? head : per) - 1);
        j.small0 = equal + tile * q;
        j.smalls = q;
        return true;
    }
};

// The jobs of the block, in order, from the planning warp to every other role;
// p0 = -1 ends a phase.
constexpr uint32_t JOB_READERS = 4 + 2;       // epilogue warps, MMA, token loader
struct JobQueue {
    int at = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void step() { if (++at == JOBS) { at = 0; phase ^= 1u; } }
    __device__ __forceinline__ static uint64_t* full(const Ctx& c, int i) { return c.full + 2 * MAX_SLOTS + 5 + i; }
    __device__ __forceinline__ static uint64_t* empty(const Ctx& c, int i) { return full(c, JOBS + i); }
    __device__ __forceinline__ static Job* job(const Ctx& c, int i) { return reinterpret_cast<Job*>(c.smem + OFF_JOBS) + i; }
    // A whole warp: its copy of the next job; false at the end of a phase, and
    // after a wait gave up (ok becomes false).
    __device__ __forceinline__ bool next(const Ctx& c, Job& j, bool& ok) {
        if (ok) ok = wait_warp(full(c, at), phase, c);
        if (!ok) return false;
        j = *job(c, at);
        const bool more = j.p0 >= 0;
        if (!more) done(c);
        return more;
    }
    // after the last use of the queue's copy of the job (or of its scales)
    __device__ __forceinline__ void done(const Ctx& c) {
        __syncwarp();
        if (c.lane == 0) mbar_arrive(empty(c, at));
        step();
    }
};

struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int slots) { if (++slot == slots) { slot = 0; phase ^= 1u; } }
};

// A slot of the ring: NP pieces of weights; the tokens' rows of each, r8
// groups of 8; their scales; MXFP4: the weights' scales.
__device__ __forceinline__ uint8_t* slot_at(const Ctx& c, int slot) { return c.smem + OFF_RING + slot * c.p.slot_bytes; }
template <int MODE> __host__ __device__ constexpr int sfb_at(int T) { return NP * (PIECE_BYTES + 1024 * rows8<MODE>(T)); }
template <int MODE> __host__ __device__ constexpr int sfa_at(int T) { return sfb_at<MODE>(T) + NP * Form<MODE>::SFB; }

// ---------------------------------------------------------------- planning and weights (one warp)

// Announces a job and loads its weights, and their scales: MXFP4 512 bytes per
// 128 rows and 128 columns, tile by tile; FP8 the UE8M0 byte of each piece,
// beside the announced job.  The bytes are on their way from HBM while the job
// is announced and its first slots are loaded: the first slot's arrival is held
// back until they are stored, which is when the MMA warp may read them.
template <int MODE>
__device__ __forceinline__ bool load_job(const Ctx& c, JobQueue& q, const Job& j, const CUtensorMap* map, const void* scales,
                                         uint64_t policy, Ring& ring) {
    constexpr int ELEMS = MODE == M_BF16 ? 64 : 128;        // map elements (bf16, or bytes) per piece
    const int words = j.k / 128;
    const size_t tile = static_cast<size_t>(j.mat) * ((j.n + 127) / 128) + j.row0 / 128;
    const uint8_t* sc = static_cast<const uint8_t*>(scales) + tile * words * 512;
    float f[JOB_PIECES / 32] = {};
    if (MODE == M_FP8) {
        const float* row = static_cast<const float*>(scales) + tile * words + j.p0;
#pragma unroll
        for (int i = 0; i < JOB_PIECES / 32; ++i)
            if (32 * i + c.lane < j.p1 - j.p0) f[i] = __ldg(row + 32 * i + c.lane);
    }
    if (!wait_warp(JobQueue::empty(c, q.at), q.phase ^ 1u, c)) return false;
    uint8_t* bytes = c.smem + OFF_JOBSC + q.at * JOB_PIECES;
    if (c.lane == 0) {
        *JobQueue::job(c, q.at) = j;
        mbar_arrive(JobQueue::full(c, q.at));
    }
    __syncwarp();
    q.step();
    uint64_t* held = c.full + ring.slot;
    // after the first two slots, or the only one
    const int store_after = MODE == M_FP8 ? min(j.p0 + NP, (j.p1 - 1) / NP * NP) : -1;
#pragma unroll 1
    for (int s = j.p0; s < j.p1; s += NP) {
        if (!wait_warp(c.empty + ring.slot, ring.phase ^ 1u, c)) return false;
        uint64_t* full = c.full + ring.slot;
        uint8_t* slot = slot_at(c, ring.slot);
        const int np = min(NP, j.p1 - s);
        const uint32_t sfa = MODE == M_FP4 ? 512u * min(2 * NP, words - 2 * s) : 0u;
        if (c.lane == 0) {
            const uint32_t tx = static_cast<uint32_t>(np * PIECE_BYTES) + sfa;
            if (MODE == M_FP8 && s == j.p0) mbar_expect_tx(full, tx);
            else mbar_arrive_expect_tx(full, tx);
            load_weights(slot, map, full, s * ELEMS, j.row0, j.mat, policy);
            if (np > 1) load_weights(slot + PIECE_BYTES, map, full, (s + 1) * ELEMS, j.row0, j.mat, policy);
            if (MODE == M_FP4) load_scales(slot + sfa_at<MODE>(c.p.T), sc + static_cast<size_t>(s) * 1024, sfa, full, policy);
        }
        __syncwarp();
        ring.next(c.p.slots);
        if (MODE == M_FP8 && s == store_after) {
#pragma unroll
            for (int i = 0; i < JOB_PIECES / 32; ++i)
                bytes[32 * i + c.lane] = static_cast<uint8_t>((__float_as_uint(f[i]) >> 23) & 0xFFu);
            __syncwarp();
            if (c.lane == 0) mbar_arrive(held);
        }
    }
    return true;
}

// Announces the end of a phase.
__device__ __forceinline__ bool end_phase(const Ctx& c, JobQueue& q) {
    if (!wait_warp(JobQueue::empty(c, q.at), q.phase ^ 1u, c)) return false;
    if (c.lane == 0) {
        JobQueue::job(c, q.at)->p0 = -1;
        mbar_arrive(JobQueue::full(c, q.at));
    }
    __syncwarp();
    q.step();
    return true;
}

// ---------------------------------------------------------------- tokens (one warp)

// Loads the tokens' rows and scales of a job's slots.
template <int MODE>
__device__ __forceinline__ bool load_tokens(const Ctx& c, const Job& j, bool third, Ring& ring) {
    const FewParams& p = c.p;
    const int r8 = rows8<MODE>(third ? __popc(j.mask) : p.T);
    const int pieces = pieces_of<MODE>(j.k);
    const uint8_t* rows = p.xq;
    const uint8_t* scales = p.xs;
    if (third) {
        rows = (j.shared ? p.hqs : p.hq) + static_cast<size_t>(j.base8) * pieces * 1024;
        scales = (j.shared ? p.hss : p.hs) + static_cast<size_t>(j.rank) * pieces * Form<MODE>::SFB;
    }
    // (a slot's second piece may lie past K: the image has it, of any contents)
    const uint32_t bytes = NP * 1024u * r8;
#pragma unroll 1
    for (int s = j.p0; s < j.p1; s += NP) {
        if (!wait_warp(c.empty + ring.slot, ring.phase ^ 1u, c)) return false;
        if (c.lane == 0) {
            uint64_t* full = c.full + ring.slot;
            uint8_t* slot = slot_at(c, ring.slot);
            mbar_arrive_expect_tx(full, bytes + NP * Form<MODE>::SFB);
            bulk_load(slot + NP * PIECE_BYTES, rows + static_cast<size_t>(s) * r8 * 1024, bytes, full);
            if (MODE != M_BF16)
                bulk_load(slot + sfb_at<MODE>(p.T), scales + static_cast<size_t>(s) * Form<MODE>::SFB, NP * Form<MODE>::SFB, full);
        }
        __syncwarp();
        ring.next(p.slots);
    }
    return true;
}

// ---------------------------------------------------------------- MMA issue (one warp)
//
// The warp runs the loop as a whole and one elected lane issues: descriptors
// and counters then are warp-uniform values (issued from a loop that only one
// lane runs, an MMA cost about 200 cycles of moves, more than it takes).

struct MmaState {
    Ring ring;
    int jobs = 0, slots = 0, rewrites = 0;
    bool leader;
    uint32_t tags = 0x100u;      // FP8, lane i: the exponent whose uniform scales are in set i
};

// FP8: the columns with the weight scale 2^(e - 127) for every row.  A set is
// rewritten when another exponent of the same residue comes up, once the MMAs
// issued before, which may read it, are done.
__device__ __forceinline__ bool uniform_scales(const Ctx& c, MmaState& st, uint32_t tmem, uint32_t e, uint32_t& cols) {
    const uint32_t set = e & 7u;
    cols = tmem + SFA_COL0 + 4 * set;
    if (__shfl_sync(0xffffffffu, st.tags, static_cast<int>(set)) == e) return true;
    uint64_t* bar = c.full + 2 * MAX_SLOTS + 4;             // the drain barrier
#pragma unroll 1
    for (int step = 0; step < 2; ++step) {                  // the MMAs before; the copy, whose source is then free
        if (step == 1) {
            const uint32_t w = e * 0x01010101u;
            reinterpret_cast<uint4*>(c.smem + OFF_UNI)[c.lane] = make_uint4(w, w, w, w);
            fence_proxy_async_smem();
            __syncwarp();
            tc_fence_after();
            if (st.leader) tmem_cp_scales(cols, c.smem + OFF_UNI);
        }
        if (st.leader) umma_commit(bar);
        __syncwarp();
        if (!wait_warp(bar, static_cast<uint32_t>(st.rewrites & 1), c)) return false;
        ++st.rewrites;
    }
    if (c.lane == static_cast<int>(set)) st.tags = e;
    return true;
}

template <int MODE>
__device__ __forceinline__ bool issue_job(const Ctx& c, const Job& j, const uint8_t* wscales, bool third, uint32_t tmem,
                                          uint64_t* accf, uint64_t* acce, MmaState& st) {
    const int buf = st.jobs & 1;
    if (!wait_warp(acce + buf, ((st.jobs >> 1) & 1) ^ 1u, c)) return false;
    tc_fence_after();
    const uint32_t d = tmem + buf * ACC_COLS;
    const int tokens = third ? __popc(__shfl_sync(0xffffffffu, j.mask, 0)) : c.p.T;
    const uint32_t n = round16(tokens * Form<MODE>::P);
    const uint32_t row_bytes = 1024u * rows8<MODE>(tokens);
    const uint32_t idesc = MODE == M_BF16 ? make_idesc(1, 128, n) : MODE == M_FP8 ? make_idesc_mxf8(128, n)
                                                                                 : make_idesc_mxf4(n, 0);
    const uint32_t idesc2 = MODE == M_FP4 ? make_idesc_mxf4(n, 2) : idesc;
    const int p0 = __shfl_sync(0xffffffffu, j.p0, 0), p1 = __shfl_sync(0xffffffffu, j.p1, 0);
    // MXFP4: the last piece of K may be a half
    const int whole = MODE == M_FP4 ? __shfl_sync(0xffffffffu, j.k, 0) / Form<MODE>::KP : p1;
#pragma unroll 1
    for (int s = p0; s < p1; s += NP) {
        if (!wait_warp(c.full + st.ring.slot, st.ring.phase, c)) return false;
        if (MODE != M_BF16 && st.slots >= 2) {
            // the MMAs that read this half of the scale columns two slots ago are done
            int q = st.ring.slot - 2;
            uint32_t ph = st.ring.phase;
            if (q < 0) { q += c.p.slots; ph ^= 1u; }
            if (!wait_warp(c.empty + q, ph, c)) return false;
        }
        uint8_t* slot = slot_at(c, st.ring.slot);
        tc_fence_after();
        const uint32_t sfb0 = tmem + SFB_COL0 + (st.slots & 1) * SFB_COLS;
        const uint32_t sfa0 = tmem + SFA_COL0 + (st.slots & 1) * SFB_COLS;
#pragma unroll
        for (int r = 0; r < NP; ++r) {
            if (s + r >= p1) break;
            uint32_t sfa = sfa0 + r * (SFB_COLS / NP);
            if (MODE == M_FP8 && !uniform_scales(c, st, tmem, wscales[s + r - p0], sfa)) return false;
            const uint64_t a = smem_desc_k_sw128(slot + r * PIECE_BYTES);
            const uint64_t b = smem_desc_k_sw128(slot + NP * PIECE_BYTES + r * row_bytes);
            const uint32_t more = s + r > p0 ? 1u : 0u;
            const uint8_t* sfb_s = slot + sfb_at<MODE>(c.p.T) + r * Form<MODE>::SFB;
            const uint8_t* sfa_s = slot + sfa_at<MODE>(c.p.T) + r * Form<MODE>::SFA;
            const uint32_t sfb = sfb0 + r * (SFB_COLS / NP);
            if (!st.leader) continue;
            if (MODE == M_BF16) {
#pragma unroll
                for (int k = 0; k < 4; ++k) umma_f16(d, a + 2 * k, b + 2 * k, idesc, more | (k > 0));
            } else if (MODE == M_FP8) {
                tmem_cp_scales(sfb, sfb_s);
#pragma unroll
                for (int k = 0; k < 4; ++k) umma_mxf8_bs(d, a + 2 * k, b + 2 * k, idesc, sfa, sfb, more | (k > 0));
            } else {
                tmem_cp_scales(sfa, sfa_s);
                tmem_cp_scales(sfb, sfb_s);
                umma_mxf4_bs(d, a, b, idesc, sfa, sfb, more);
                umma_mxf4_bs(d, a + 2, b + 2, idesc2, sfa, sfb, 1);
                if (s + r < whole) {
                    tmem_cp_scales(sfa + 4, sfa_s + 512);
                    tmem_cp_scales(sfb + 4, sfb_s + 512);
                    umma_mxf4_bs(d, a + 4, b + 4, idesc, sfa + 4, sfb + 4, 1);
                    umma_mxf4_bs(d, a + 6, b + 6, idesc2, sfa + 4, sfb + 4, 1);
                }
            }
        }
        __syncwarp();
        ++st.slots;
        if (st.leader) umma_commit(c.empty + st.ring.slot);
        st.ring.next(c.p.slots);
    }
    if (st.leader) umma_commit(accf + buf);
    __syncwarp();
    ++st.jobs;
    return true;
}

// ---------------------------------------------------------------- epilogue (128 threads, thread = row)

// Adds a job's products to the thread's sums: out[t * 128] += gate * (v + bias).
template <int MODE>
__device__ __forceinline__ void read_job(const Ctx& c, const Job& j, bool third, float bias, uint32_t tmem, uint64_t* accf,
                                         uint64_t* acce, int& jobs, bool& ok, float* out) {
    const int buf = jobs & 1;
    if (ok) ok = wait_warp(accf + buf, (jobs >> 1) & 1, c);
    ++jobs;
    if (!ok) return;
    tc_fence_after();
    const uint32_t acc = tmem + (static_cast<uint32_t>(c.warp * 32) << 16) + buf * ACC_COLS;
    const bool gated = third && !j.shared;
    auto add = [&](int t, float v) {
        const float g = gated ? reinterpret_cast<const float*>(c.smem + OFF_GATE)[t * 16 + (static_cast<int>(j.kpack >> (4 * t)) & 15)]
                              : 1.f;
        out[t * 128] = fmaf(g, v + bias, out[t * 128]);
    };
    // phase 2: token t's columns are t P ..; phase 3: those of its place in the mask
    if (Form<MODE>::P == 1) {
        uint32_t r[16];
        tmem_ld_32x32b_x16(acc, r);
        tmem_ld_wait_regs(r);
        tc_fence_before();
        mbar_arrive(acce + buf);
        uint32_t m = third ? j.mask : (1u << c.p.T) - 1u;
#pragma unroll
        for (int i = 0; i < MAX_T; ++i) {
            if (!m) break;
            const int t = __ffs(m) - 1;
            m &= m - 1;
            if (j.mask >> t & 1u) add(t, __uint_as_float(r[i]));
        }
    } else {
        // five columns a token (the load reads three more)
        int i = 0;
#pragma unroll 1
        for (uint32_t m = j.mask; m; m &= m - 1, ++i) {
            const int t = __ffs(m) - 1;
            uint32_t r[8];
            tmem_ld_32x32b_x8(acc + static_cast<uint32_t>(PLANES * (third ? i : t)), r);
            tmem_ld_wait_regs(r);
            float v = __uint_as_float(r[PLANES - 1]);
#pragma unroll
            for (int q = PLANES - 2; q >= 0; --q) v += __uint_as_float(r[q]);
            add(t, v);
        }
        tc_fence_before();
        mbar_arrive(acce + buf);
    }
}

// A tile that crosses shares: stores this share's sums (out_s[t * 128 + row],
// the tokens of `mask`), and in the last of the tile's shares to get here
// replaces them by the total, in the order of the shares.  True where the sums
// are now the tile's.  Every epilogue thread calls it.
__device__ __forceinline__ bool combine(const Ctx& c, const Job& j, uint32_t mask, float* out_s) {
    const FewParams& p = c.p;
    const int parts = j.share1 - j.share0 + 1 + j.smalls;
    if (parts == 1) return true;
    // a share has at most one tile it continues and one it leaves unfinished
    auto part = [&](int s) { return p.sums + (static_cast<size_t>(s) * 2 + (s == j.share0)) * p.T * 128; };
    float* mine = part(j.share);
#pragma unroll 1
    for (uint32_t m = mask; m; m &= m - 1) {
        const int at = (__ffs(m) - 1) * 128 + c.tid;
        __stcg(mine + at, out_s[at]);
    }
    int* last_s = reinterpret_cast<int*>(c.smem + OFF_MISC) + 3;
    bar_epilogue();
    if (c.tid == 0) {
        uint32_t* ctr = p.ctr + CTR_TILE + j.share0;
        const bool last = add_acq_rel(ctr) == static_cast<uint32_t>(parts - 1);
        if (last) *ctr = 0;
        *last_s = last;
    }
    bar_epilogue();
    if (!*last_s) {
        bar_epilogue();                                        // the flag may be written again
        return false;
    }
    // four rows of a token a thread, up to four tokens, a few parts at a time
    float4 v[MAX_T / 4];
#pragma unroll
    for (int q = 0; q < MAX_T / 4; ++q) v[q] = make_float4(0.f, 0.f, 0.f, 0.f);
    const uint32_t mine4 = mask >> c.warp;                     // bit 4 q: the q-th token of the warp
#pragma unroll 4
    for (int x = 0; x < parts; ++x) {
        const int s = j.share0 + x <= j.share1 ? j.share0 + x : j.small0 + x - (j.share1 - j.share0 + 1);
        const float4* src = reinterpret_cast<const float4*>(part(s)) + c.tid;
#pragma unroll
        for (int q = 0; q < MAX_T / 4; ++q)
            if (mine4 >> (4 * q) & 1u) {
                const float4 w = __ldcg(src + q * EPI);
                v[q].x += w.x; v[q].y += w.y; v[q].z += w.z; v[q].w += w.w;
            }
    }
#pragma unroll
    for (int q = 0; q < MAX_T / 4; ++q)
        if (mine4 >> (4 * q) & 1u) reinterpret_cast<float4*>(out_s)[q * EPI + c.tid] = v[q];
    bar_epilogue();
    return true;
}

// ---------------------------------------------------------------- phase 1

// (A warp holds an expert's slice in registers, 14 float4 a lane in one round of
// loads, and runs the tokens past it.)
template <int MODE>
__device__ __forceinline__ void router_and_x(const Ctx& c) {
    const FewParams& p = c.p;
    // a block has one slice of d and a share of the experts; it stages the
    // tokens' slices in the ring's memory
    const int sharers = gridDim.x / p.ks, who = blockIdx.x / p.ks, ks = blockIdx.x % p.ks;
    __nv_bfloat16* xsm = reinterpret_cast<__nv_bfloat16*>(c.smem + OFF_RING);
    const int e0 = p.E * who / sharers, e1 = p.E * (who + 1) / sharers;
    if (who < sharers && e0 < e1) {
        const int k0 = ks * p.slice, len = min(p.slice, p.d - k0);       // multiples of 64
        // a token's slice and zeros up to the width that a warp computes
        constexpr int W8 = SLICE_PIECES * 16;
#pragma unroll 1
        for (int i = c.tid; i < p.T * W8; i += CT) {
            const int t = i / W8, q = i - t * W8;
            uint4* dst = reinterpret_cast<uint4*>(xsm) + i;
            if (8 * q < len) cp_async_16(dst, reinterpret_cast<const uint4*>(p.x + static_cast<size_t>(t) * p.d + k0) + q);
            else *dst = make_uint4(0, 0, 0, 0);
        }
#pragma unroll 1
        for (int e = e0 + c.warp; e < e0 + (e1 - e0 + CW - 1) / CW * CW; e += CW) {
            float4 w[SLICE_PIECES];
            const float4* src = reinterpret_cast<const float4*>(p.W_r + static_cast<size_t>(min(e, p.E - 1)) * p.d + k0);
#pragma unroll
            for (int i = 0; i < SLICE_PIECES; ++i)
                w[i] = 32 * i + c.lane < len / 4 ? __ldg(src + 32 * i + c.lane) : make_float4(0.f, 0.f, 0.f, 0.f);
            if (e < e0 + CW) {                                           // the slices of x are there
                asm volatile("cp.async.wait_all;" ::: "memory");
                bar_general();
            }
            if (e >= e1) continue;
#pragma unroll 1
            for (int t = 0; t < p.T; ++t) {
                const uint2* xt = reinterpret_cast<const uint2*>(xsm) + t * (2 * W8) + c.lane;
                float acc[4] = {};                                       // one per element of a float4
#pragma unroll
                for (int i = 0; i < SLICE_PIECES; ++i) {
                    const uint2 xv = xt[32 * i];
                    acc[0] = fmaf(__uint_as_float(xv.x << 16), w[i].x, acc[0]);
                    acc[1] = fmaf(__uint_as_float(xv.x & 0xFFFF0000u), w[i].y, acc[1]);
                    acc[2] = fmaf(__uint_as_float(xv.y << 16), w[i].z, acc[2]);
                    acc[3] = fmaf(__uint_as_float(xv.y & 0xFFFF0000u), w[i].w, acc[3]);
                }
                float v = (acc[0] + acc[1]) + (acc[2] + acc[3]);
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
                if (c.lane == 0) p.part[(static_cast<size_t>(ks) * p.T + t) * p.e4 + e] = v;
            }
        }
    }
    // the image of x, a warp per 128 columns (bf16: d may end inside them)
    const int nb = (p.d + 127) / 128;
#pragma unroll 1
    for (int i = blockIdx.x * CW + c.warp; i < p.T * nb; i += gridDim.x * CW) {
        const int t = i / nb, col = (i - t * nb) * 128;
        uint2 raw = make_uint2(0, 0);
        if (MODE != M_BF16 || col + 4 * c.lane < p.d)
            raw = __ldg(reinterpret_cast<const uint2*>(p.x + static_cast<size_t>(t) * p.d + col) + c.lane);
        store_block<MODE>(make_float4(__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xFFFF0000u),
                                      __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xFFFF0000u)),
                          p.xq, p.xs, rows8<MODE>(p.T), t, col, c.lane);
    }
    fence_proxy_async_all();                                   // read by bulk copies after the barrier
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
template <int MODE>
__device__ __forceinline__ void select_experts(const Ctx& c) {
    const FewParams& p = c.p;
    int* idx_s = reinterpret_cast<int*>(c.smem + OFF_IDX);
    float* gate_s = reinterpret_cast<float*>(c.smem + OFF_GATE);
    uint32_t* mask_s = reinterpret_cast<uint32_t*>(c.smem + OFF_MASK);
    uint64_t* kpack_s = reinterpret_cast<uint64_t*>(c.smem + OFF_KPACK);
    int* act_s = reinterpret_cast<int*>(c.smem + OFF_ACT);
    int* misc = reinterpret_cast<int*>(c.smem + OFF_MISC);
    const bool writer = blockIdx.x == gridDim.x - 1;
    // the partial logits into the ring's memory at once (read by every block:
    // a dependent read of the same few lines by all of them costs 2 us each)
    float* part_s = reinterpret_cast<float*>(c.smem + OFF_RING);
    const int chunk = min(p.T, static_cast<int>(RING_BYTES / 4) / (p.ks * p.e4));  // tokens that fit
#pragma unroll 1
    for (int t0 = 0; t0 < p.T; t0 += chunk) {
        const int nt = min(chunk, p.T - t0), row = nt * p.e4 / 4;                  // float4 per slice
        bar_general();
#pragma unroll 1
        for (int i = c.tid; i < p.ks * row; i += CT) {
            const int s = i / row;
            cp_async_16(part_s + 4 * i, p.part + (static_cast<size_t>(s) * p.T + t0) * p.e4 + 4 * (i - s * row));
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        bar_general();
#pragma unroll 1
        for (int t = t0 + c.warp; t < t0 + nt; t += CW) {
        float l[8];
        uint32_t key[8];
        float top = -INFINITY;
        const float* part = part_s + (t - t0) * p.e4;
#pragma unroll
        for (int i = 0; i < 8; ++i) l[i] = 0.f;
#pragma unroll 2
        for (int s = 0; s < p.ks; ++s) {
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] += part[s * 4 * row + min(32 * i + c.lane, p.E - 1)];
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
        float best_l = -INFINITY, mine = 0.f;
#pragma unroll 1
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
            best_l = fmaxf(best_l, v);
            if (c.lane == k) mine = v;
            if (c.lane == 0) idx_s[t * 16 + k] = static_cast<int>(e);
        }
        // gates: relative to the largest logit chosen, which a bias on the
        // selection alone may leave far below the largest of all
        mine = c.lane < p.K ? expf(mine - best_l) : 0.f;
        float chosen = 0.f;
#pragma unroll 4
        for (int k = 0; k < p.K; ++k) chosen += __shfl_sync(0xffffffffu, mine, k);
        if (c.lane < p.K) gate_s[t * 16 + c.lane] = mine / chosen;
        if (writer) {
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
            const float inv = 1.f / sum;
#pragma unroll
            for (int i = 0; i < 8; ++i) p.prob[t * 256 + 32 * i + c.lane] = l[i] * inv;
        }
        }
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
#pragma unroll 1
        for (int k = 0; k < (p.slot_major ? p.K : 1); ++k)
#pragma unroll 1
            for (uint32_t m = mask; m && left > 0; m &= m - 1) {
                const int t = __ffs(m) - 1;
                if (!p.slot_major || (static_cast<int>(kpack >> (4 * t)) & 15) == k) { keep |= 1u << t; --left; }
            }
        mask = keep;
        mask_s[e] = keep;
    }
    // experts reached, in ascending order, and where their images of h start
    const uint32_t votes = __ballot_sync(0xffffffffu, mask != 0);
    const int r8 = rows8<MODE>(__popc(mask));
    int before = r8;                                           // inclusive sum over the warp
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (c.lane >= o) before += v;
    }
    if (c.lane == 31) {
        misc[4 + c.warp] = __popc(votes);
        misc[12 + c.warp] = before;
    }
    bar_general();
    int rank = __popc(votes & ((1u << c.lane) - 1u)), base8 = before - r8, total = 0;
#pragma unroll
    for (int w = 0; w < CW; ++w) {
        if (w < c.warp) {
            rank += misc[4 + w];
            base8 += misc[12 + w];
        }
        total += misc[4 + w];
    }
    if (mask) {
        act_s[rank] = e;
        reinterpret_cast<int*>(c.smem + OFF_BASE)[e] = base8 | rank << 16;
    }
    if (c.tid == 0) misc[1] = total;
}

// The routing outputs and the balance statistics, by warps 4..7 of the last
// block, which have nothing to do in phase 3.
__device__ __forceinline__ void balance(const Ctx& c) {
    const FewParams& p = c.p;
    const int i = c.tid - EPI;
#pragma unroll 1
    for (int s = i; s < p.T * p.K; s += EPI) {
        const int at = s / p.K * 16 + s % p.K;
        if (p.topk_idx) p.topk_idx[s] = reinterpret_cast<const int*>(c.smem + OFF_IDX)[at];
        if (p.gates) p.gates[s] = reinterpret_cast<const float*>(c.smem + OFF_GATE)[at];
    }
    float sum = 0.f;
#pragma unroll 1
    for (int e = i; e < p.E; e += EPI) {
        float P = 0.f;
#pragma unroll 1
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
    float* red = reinterpret_cast<float*>(c.smem + OFF_MISC) + 4;              // (the selection is over)
    if (c.lane == 0) red[c.warp - 4] = sum;
    bar_upper();
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
    int* misc = reinterpret_cast<int*>(smem + OFF_MISC);
    const Ctx c{p, smem, full, full + MAX_SLOTS, misc, static_cast<int>(threadIdx.x),
                static_cast<int>(threadIdx.x >> 5), static_cast<int>(threadIdx.x & 31)};
    if (c.tid == 0) {
        for (int i = 0; i < MAX_SLOTS; ++i) {
            mbar_init(c.full + i, 2);                           // weights, tokens
            mbar_init(c.empty + i, 1);
        }
        for (int i = 0; i < 2; ++i) { mbar_init(accf + i, 1); mbar_init(acce + i, EPI); }
        mbar_init(full + 2 * MAX_SLOTS + 4, 1);
        for (int i = 0; i < JOBS; ++i) {
            mbar_init(JobQueue::full(c, i), 1);
            mbar_init(JobQueue::empty(c, i), JOB_READERS);
        }
        misc[0] = 0;
        fence_mbar_init();
    }
    if (c.warp == W_MMA) tmem_alloc<TMEM_COLS>(reinterpret_cast<uint32_t*>(misc + 2));
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(misc[2]);

    if (c.warp == W_LOAD) {
        if (c.lane == 0) {
            tma_prefetch_desc(&p.w1);
            tma_prefetch_desc(&p.w2);
            if (p.S) { tma_prefetch_desc(&p.ws1); tma_prefetch_desc(&p.ws2); }
        }
        __syncthreads();                                        // the experts are selected
        const int n_active = misc[1];
        const uint64_t policy = evict_first_policy();
        Ring ring;
        JobQueue queue;
        bool ok = *c.abort_flag == 0;
        Job j;
#pragma unroll 1
        for (int phase = 2; phase <= 3; ++phase) {
            const bool third = phase == 3;
            Plan<MODE> plan(c, phase, n_active);
            // the first share is the block's own, the others come off a counter,
            // drawn a share ahead
            int share = blockIdx.x;
#pragma unroll 1
            while (ok && share < plan.shares) {
                int after = 0;
                if (c.lane == 0) after = static_cast<int>(gridDim.x + atomicAdd(p.ctr + CTR_SHARE + phase - 2, 1u));
                plan.take(share);
#pragma unroll 1
                while (ok && plan.next(j)) {
                    const void* sc = third ? (j.shared ? p.ws2s : p.w2s) : (j.shared ? p.ws1s : p.w1s);
                    ok = load_job<MODE>(c, queue, j, third ? (j.shared ? &p.ws2 : &p.w2) : (j.shared ? &p.ws1 : &p.w1), sc,
                                        policy, ring);
                }
                share = __shfl_sync(0xffffffffu, after, 0);
            }
            ok = ok && end_phase(c, queue);
        }
        // a block that gave up leaves its copies the time to land before it
        // gives its memory back (their barriers may never complete)
        if (!ok && c.lane == 0) {
            const uint64_t t0 = global_timer_ns();
            while (global_timer_ns() - t0 < kDrainNs) {}
        }
        __syncwarp();
    } else if (c.warp == W_TOKENS) {
        __syncthreads();
        Ring ring;
        JobQueue queue;
        bool ok = *c.abort_flag == 0;
        Job j;
#pragma unroll 1
        for (int phase = 2; phase <= 3; ++phase) {
            if (phase == 3) bar_tokens_ready();
            fence_proxy_async_all();                            // the images were written through the generic proxy
            while (queue.next(c, j, ok)) {
                queue.done(c);
                ok = load_tokens<MODE>(c, j, phase == 3, ring);
            }
        }
    } else if (c.warp == W_MMA) {
        __syncthreads();
        MmaState st;
        st.leader = elect_one();
        JobQueue queue;
        bool ok = *c.abort_flag == 0;
        Job j;
#pragma unroll 1
        for (int phase = 2; phase <= 3; ++phase)
            while (queue.next(c, j, ok)) {
                ok = issue_job<MODE>(c, j, smem + OFF_JOBSC + queue.at * JOB_PIECES, phase == 3, tmem, accf, acce, st);
                queue.done(c);
            }
        if (!ok && st.leader) {
            umma_commit(full + 2 * MAX_SLOTS + 4);
            volatile int no_abort = 0;
            mbar_wait_bounded(full + 2 * MAX_SLOTS + 4, static_cast<uint32_t>(st.rewrites & 1), &no_abort, nullptr, kDrainNs);
        }
        __syncwarp();
    } else {
        router_and_x<MODE>(c);
        grid_barrier(p.ctr, 0, p.status, c.abort_flag, c.tid);
        select_experts<MODE>(c);
        fence_proxy_async_smem();                               // phase 1 used the ring's memory
        __syncthreads();
        const int* idx_s = reinterpret_cast<const int*>(smem + OFF_IDX);
        const float* gate_s = reinterpret_cast<const float*>(smem + OFF_GATE);
        const uint32_t* mask_s = reinterpret_cast<const uint32_t*>(smem + OFF_MASK);
        float* out_s = reinterpret_cast<float*>(smem + OFF_OUT);                   // [T][128]
        float* sums = out_s + c.tid;                                               // epilogue: this thread's row
        JobQueue queue;
        int jobs_read = 0;
        bool ok = *c.abort_flag == 0;
#pragma unroll 1
        for (int phase = 2; phase <= 3; ++phase) {
            const bool third = phase == 3;
            if (third) {
                fence_proxy_async_all();                        // phase 2 wrote the image of h
                grid_barrier(p.ctr, 1, p.status, c.abort_flag, c.tid);
                bar_tokens_ready();
                ok = ok && *c.abort_flag == 0;
            }
            if (c.warp >= 4) {
                if (third && blockIdx.x == gridDim.x - 1) balance(c);
                continue;
            }
            bool begins = true;
            Job j;
            while (true) {
                const bool got = queue.next(c, j, ok);
                const int row = j.row0 + c.tid;
                const bool in = got && row < j.n;
                float bias = 0.f;
                if (got) {
                    queue.done(c);
                    if (begins) {
#pragma unroll 1
                        for (int t = 0; t < p.T; ++t) sums[t * 128] = 0.f;
                    }
                    begins = j.ends;
                    // phase 3: the share with a matrix's first piece adds its bias
                    const float* biases = third ? (j.shared ? p.bs2 : p.b2) : (j.shared ? p.bs1 : p.b1);
                    if (in && (!third || j.p0 == 0)) bias = __ldg(biases + static_cast<size_t>(j.mat) * j.n + row);
                    read_job<MODE>(c, j, third, third ? bias : 0.f, tmem, accf, acce, jobs_read, ok, sums);
                }
                // a wait that gave up ends the phase for the four warps together:
                // what follows has barriers between them
                ok = all_ok(ok);
                if (!ok || !got) break;
                const uint32_t tokens = third ? (1u << p.T) - 1u : j.mask;
                if (!j.ends || !combine(c, j, tokens, out_s)) continue;
                if (!third) {
                    uint8_t* rows = (j.shared ? p.hqs : p.hq) + static_cast<size_t>(j.base8) * pieces_of<MODE>(j.n) * 1024;
                    uint8_t* scales = (j.shared ? p.hss : p.hs) + static_cast<size_t>(j.rank) * pieces_of<MODE>(j.n) * Form<MODE>::SFB;
                    const int r8 = rows8<MODE>(__popc(j.mask));
#pragma unroll 1
                    for (uint32_t m = tokens; m; m &= m - 1) {
                        const int t = __ffs(m) - 1;
                        const float h = silu_fast(sums[t * 128] + bias);
                        if (MODE == M_BF16) {
                            // two bytes of row (the token's place) of a piece
                            if (!in) continue;
                            const int n = column_of(j, t), at = 2 * row;
                            uint8_t* dst = rows + (static_cast<size_t>(at >> 7) * r8 + (n >> 3)) * 1024 + (n & 7) * 128 +
                                           ((((at >> 4) & 7) ^ (n & 7)) << 4) + (at & 15);
                            *reinterpret_cast<__nv_bfloat16*>(dst) = __float2bfloat16_rn(h);
                        } else {
                            sums[t * 128] = h;
                        }
                    }
                    if (MODE != M_BF16) {
                        // the tile's rows are 128 columns of h, which a warp per token writes
                        bar_epilogue();
                        int i = 0;
#pragma unroll 1
                        for (uint32_t m = tokens; m; m &= m - 1, ++i) {
                            const int t = __ffs(m) - 1;
                            if ((i & 3) == c.warp)
                                store_block<MODE>(reinterpret_cast<const float4*>(out_s + t * 128)[c.lane], rows, scales, r8, i,
                                                  j.row0, c.lane);
                        }
                        bar_epilogue();
                    }
                    continue;
                }
                if (!in) continue;
#pragma unroll 1
                for (uint32_t m = tokens; m; m &= m - 1) {
                    const int t = __ffs(m) - 1;
                    float v = sums[t * 128];
                    const size_t at = static_cast<size_t>(t) * p.d + row;
                    if (p.passthrough) {
#pragma unroll 1
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
    // the last block to leave zeroes the counters for the next launch (a
    // tile's own are zero again unless a block gave up)
    if (c.tid == 0) {
        if (*c.abort_flag) atomicExch(p.ctr + CTR_ABORT, 1u);
        __threadfence();
        if (atomicAdd(p.ctr + CTR_EXIT, 1u) == gridDim.x - 1) {
            __threadfence();
            if (ld_acquire(p.ctr + CTR_ABORT))
#pragma unroll 1
                for (unsigned i = 0; i < SHARES * gridDim.x; ++i) p.ctr[CTR_TILE + i] = 0;
#pragma unroll 1
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
    size_t ctr, part, prob, xq, xs, hq, hs, hqs, hss, sums, total;
};

// blocks: as many as can find work, at most one per SM
struct FewPlan {
    int blocks, ks, slice;
};

FewPlan few_plan(const Dims& dm, int sms) {
    FewPlan f;
    if (sms > MAX_BLOCKS) sms = MAX_BLOCKS;
    // a block per slot of weights that the most experts reached would have
    const long long reached = dm.T * dm.K < dm.E ? dm.T * dm.K : dm.E;
    auto slots = [&](long long rows, int k) {
        return (rows + 127) / 128 * (dm.dtype == MOE_BF16 ? slots_of<M_BF16>(k) : dm.dtype == MOE_MXFP4 ? slots_of<M_FP4>(k)
                                                                                                     : slots_of<M_FP8>(k));
    };
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

template <int MODE>
FewLayout few_layout_mode(const Dims& dm) {
    FewLayout L{};
    size_t off = 0;
    auto take = [&](size_t bytes) { const size_t o = off; off = align256(off + bytes); return o; };
    auto pieces = [](int k) { return static_cast<size_t>(pieces_of<MODE>(k)); };
    take(256);                                              // status word
    L.ctr = take((CTR_TILE + SHARES * MAX_BLOCKS) * 4);
    // slices are at least 128 columns long, whatever the device's size
    L.part = take(static_cast<size_t>((dm.d + 127) / 128) * dm.T * ((dm.E + 3) & ~3) * 4);
    L.prob = take(static_cast<size_t>(dm.T) * 256 * 4);
    // images: the groups of 8 rows of T K slots over the experts reached are
    // at most (T K P + 7 experts) / 8
    const size_t reached = dm.T * dm.K < dm.E ? dm.T * dm.K : dm.E;
    const size_t groups = (static_cast<size_t>(dm.T) * dm.K * Form<MODE>::P + 7 * reached) / 8;
    L.xq = take(pieces(dm.d) * rows8<MODE>(dm.T) * 1024);
    L.xs = take(pieces(dm.d) * Form<MODE>::SFB);
    L.hq = take(pieces(dm.dff) * groups * 1024);
    L.hs = take(pieces(dm.dff) * reached * Form<MODE>::SFB);
    L.hqs = take(pieces(dm.dffs) * dm.S * rows8<MODE>(dm.T) * 1024);
    L.hss = take(pieces(dm.dffs) * dm.S * Form<MODE>::SFB);
    L.sums = take(static_cast<size_t>(SHARES) * MAX_BLOCKS * 2 * dm.T * 128 * 4);
    L.total = off;
    return L;
}

FewLayout few_layout(const Dims& dm) {
    return dm.dtype == MOE_BF16 ? few_layout_mode<M_BF16>(dm)
           : dm.dtype == MOE_MXFP4 ? few_layout_mode<M_FP4>(dm) : few_layout_mode<M_FP8>(dm);
}

template <int MODE>
cudaError_t launch_mode(FewParams& p, int blocks, cudaStream_t st) {
    static_assert(RING_BYTES / (sfa_at<MODE>(MAX_T) + NP * Form<MODE>::SFA) >= 3, "two slots of MMAs in flight");
    p.slot_bytes = sfa_at<MODE>(p.T) + NP * Form<MODE>::SFA;
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
    p.xq = w + L.xq;
    p.xs = w + L.xs;
    p.hq = w + L.hq;
    p.hs = w + L.hs;
    p.hqs = w + L.hqs;
    p.hss = w + L.hss;
    p.sums = reinterpret_cast<float*>(w + L.sums);
    p.alpha = dm.alpha;
    p.T = dm.T;
    p.d = dm.d;
    p.E = dm.E;
    p.e4 = (dm.E + 3) & ~3;
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
